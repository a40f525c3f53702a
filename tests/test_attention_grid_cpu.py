"""C ABI of attention backward: sizes whose launches would have more than 2^31 - 1 blocks are refused."""
import ctypes

import pytest

import exact_sum_gemm_gb300 as dg
from exact_sum_gemm_gb300 import _native

SHAPE = 3
F32, BF16 = 0, 1


def backward(dtype, **sizes):
    a = dict(batch=1, lq=1, lk=1, hq=1, hkv=1, dim=8, scale=0.1, causal=0, k_lengths=None)
    a.update(sizes)
    h = _native.Heads(16, 8, 8, 8)
    shape = _native.AttentionShape(*a.values())
    return dg.library().det_attention_backward(dtype, ctypes.byref(shape), h, h, h, h, h, 16, h, h, h, None)


# bf16: 8 blocks of 16 queries per 128 of a head; both: a block per 64 queries and per 64 keys
@pytest.mark.parametrize("dtype,sizes", [
    (BF16, dict(batch=1 << 13, hq=1 << 15, hkv=1)),                    # 2^31 blocks of queries
    (BF16, dict(batch=1 << 12, hq=1 << 15, hkv=1, lq=129)),
    (F32, dict(batch=1 << 15, hq=1 << 15, hkv=1 << 15)),               # 2^30 of queries, 2^30 of keys
    (BF16, dict(batch=1 << 15, hq=1 << 15, hkv=1 << 15)),
])
def test_too_many_blocks(dtype, sizes):
    assert backward(dtype, **sizes) == SHAPE
