"""The extension behind the serving calls without a GPU: what does not fit
comes back as None with nothing enqueued, and qar.py says why."""
import os

import pytest
import torch

from block_wise_int8_amd import qar

I32 = torch.int32


@pytest.fixture(scope="module")
def ext():
    return qar._serve()


def _cache():
    return qar.KvCache.empty(4, 2, 64, 2, 2, device="cpu")


def test_it_is_in_the_tree(ext):
    assert os.path.realpath(ext.__file__) == os.path.realpath(qar.EXTENSION)


def test_arguments_are_counted(ext):
    for name, count in (("kv8_append", 4), ("kv8_read", 5), ("kv8_attention", 7), ("kv8_evict", 7), ("mx4_quantize", 3),
                        ("mx4_dequantize", 5), ("mx4_linear", 6)):
        for wrong in (0, count - 1, count + 1):
            with pytest.raises(TypeError, match=f"{count} arguments"):
                getattr(ext, name)(*[None] * wrong)
        assert getattr(ext, name)(*[None] * count) is None


def test_host_tensors_and_other_objects_come_back(ext):
    c, starts, x = _cache(), torch.zeros(2, dtype=I32), torch.zeros((2, 1, 2, 64))
    assert ext.kv8_append(c, starts, x, x) is None
    assert ext.kv8_read(c, starts, 1, torch.float32, None) is None
    assert ext.kv8_read(c, starts, 1 << 70, torch.float32, None) is None
    assert ext.kv8_attention(c, x, None, None, None, None, None) is None
    assert ext.kv8_evict(c, c, torch.zeros((2, 2, 128)), 1, 1, None, None) is None
    assert ext.mx4_quantize(torch.zeros(2, 32), None, None) is None
    for broken in (object(), None, 3, qar.KvCache(None, *[starts] * 5), qar.KvCache(*[starts] * 6)):
        assert ext.kv8_append(broken, starts, x, x) is None


def test_the_reasons():
    c, starts = _cache(), torch.zeros(2, dtype=I32)
    with pytest.raises(TypeError, match="cache.k must be a CUDA"):
        qar.qar_kv8_append(c, starts, torch.zeros((2, 1, 2, 64)), torch.zeros((2, 1, 2, 64)))
    with pytest.raises(TypeError, match="cache.v must be a CUDA"):
        qar.qar_kv8_read(qar.KvCache(c.k, c.k_scales, None, c.v_scales, c.page_table, c.lengths), starts, 1)
    with pytest.raises(ValueError, match="cols must be"):
        qar.qar_mx4_dequantize(torch.zeros((2, 16), dtype=torch.uint8), torch.zeros((2, 1), dtype=torch.uint8), -1)
    with pytest.raises(TypeError, match="x must be a CUDA"):
        qar.qar_mx4_linear(None, None, None)
