"""C ABI of the training operators: strides whose byte offsets would pass 63 bits are refused."""
import ctypes

import exact_sum_gemm_gb300 as dg
from exact_sum_gemm_gb300 import _native

INVALID = 1
FAR = 1 << 40                                               # the largest stride


def test_rows():
    lib = dg.library()
    rows = 1 << 30
    norm = lambda ldx, ldy: lib.det_layer_norm_forward(0, 0, rows, 4, 16, ldx, None, None, 1e-5, 16, ldy, 4, 4, None)  # noqa: E731
    assert norm(FAR, 4) == INVALID and norm(4, FAR) == INVALID
    back = lambda lddy, ldx, lddx: lib.det_layer_norm_backward(0, 0, rows, 4, 16, lddy, 16, ldx, 4, 4, None, 16,  # noqa: E731
                                                               lddx, None, None, None)
    assert back(FAR, 4, 4) == INVALID and back(4, FAR, 4) == INVALID and back(4, 4, FAR) == INVALID
    assert lib.det_token_logprobs_forward(1, rows, 10, 16, FAR, 8, 0, 4, 4, 4, 4, 8, None) == INVALID
    assert lib.det_token_logprobs_backward(1, rows, 10, 4, 4, 16, FAR, 8, 4, 4, 16, 10, None) == INVALID
    assert lib.det_token_logprobs_backward(1, rows, 10, 4, 4, 16, 10, 8, 4, 4, 16, FAR, None) == INVALID


def test_heads():
    shape = _native.AttentionShape(1 << 20, 64, 64, 64, 64, 64, 0.1, 0, None)
    good = _native.Heads(16, 64 * 64 * 64, 64 * 64, 64)
    far = _native.Heads(16, FAR, 64 * 64, 64)               # 2^60 elements to the last entry
    call = lambda *h: dg.library().det_attention_forward(1, ctypes.byref(shape), *h, 16, None)  # noqa: E731
    for i in range(4):
        assert call(*(far if i == j else good for j in range(4))) == INVALID, i
