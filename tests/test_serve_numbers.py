"""Whole numbers among the serving calls' arguments: Python's and NumPy's are taken, truth values, tensors and others refused,
the same by the extension and by the checks behind it."""
import numpy as np
import pytest
import torch

from block_wise_int8_amd import qar

WHOLE = [5, np.int64(5), np.int32(5), np.uint8(5)]
NOT_WHOLE = [True, 5.0, np.float32(5), torch.tensor(5), "5", -5, np.int64(-5), 1 << 70]


@pytest.mark.parametrize("v", WHOLE, ids=lambda v: type(v).__name__)
def test_taken(v):
    qar._whole(v, "tokens", 0, 1 << 32)


@pytest.mark.parametrize("v", NOT_WHOLE, ids=lambda v: f"{type(v).__name__}")
def test_refused(v):
    with pytest.raises(ValueError, match="tokens must be a whole number"):
        qar._whole(v, "tokens", 0, 1 << 32)


@pytest.mark.gpu
def test_calls():
    """Equal results for equal numbers of any such type; everything else raises."""
    dev = "cuda:0"
    g = torch.Generator(device=dev).manual_seed(0)
    cache = qar.KvCache.empty(4, 2, 64, 1, 2)
    cache.page_table.copy_(torch.tensor([[2, 0]], dtype=torch.int32))
    into = qar.KvCache.empty(4, 2, 64, 1, 1)
    into.page_table.fill_(1)
    x = torch.randn((1, 100, 2, 64), generator=g, device=dev)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    qar.qar_kv8_append(cache, zero, x, -x)
    cache.lengths += 100
    w = torch.rand((1, 2, 128), generator=g, device=dev)
    codes, scales = qar.qar_mx4_quantize(x.view(200, 64))
    want = qar.qar_kv8_read(cache, zero, 5), qar.qar_kv8_evict(cache, into, w, 5, 50), qar.qar_mx4_dequantize(codes, scales, 64)
    for v in WHOLE:
        assert all(torch.equal(a, b) for a, b in zip(qar.qar_kv8_read(cache, zero, v), want[0]))
        assert all(torch.equal(a, b) for a, b in zip(qar.qar_kv8_evict(cache, into, w, v, type(v)(50)), want[1]))
        assert torch.equal(qar.qar_mx4_dequantize(codes, scales, type(v)(64)), want[2])
    for v in NOT_WHOLE:
        for call in (lambda: qar.qar_kv8_read(cache, zero, v), lambda: qar.qar_kv8_evict(cache, into, w, 5, v),
                     lambda: qar.qar_kv8_evict(cache, into, w, v, 50), lambda: qar.qar_mx4_dequantize(codes, scales, v)):
            with pytest.raises((ValueError, TypeError)):
                call()
