"""Calls around forked sequences whose launches would pass 2^32 threads are refused, without a GPU (nothing is launched)."""
import ctypes

import pytest
from test_fork_abi import NEW, _calls
from test_serve_abi import INV, M, _struct

from block_wise_int8_amd import qar


@pytest.fixture(scope="module")
def L():
    return qar.lib()


def test_sequences(L):
    """A workgroup of 256 for each of 2^24."""
    fork, free, reserve, compact, _ = _calls(L)
    many = dict(batch=1 << 24, table_width=1)
    for call in (free, reserve, compact):
        assert call(ctypes.byref(_struct(**many))) == INV
    into = ctypes.byref(_struct(**{**NEW, **many}))
    assert fork(ctypes.byref(_struct(table_width=1)), into) == INV
    assert fork(ctypes.byref(_struct(**many)), ctypes.byref(_struct(**{**NEW, "table_width": 1}))) == INV


def test_attention_behind_shared_prefixes(L):
    """dim / 4 threads join a row of outputs: 2^30 / dim * 16 rows are 2^32 threads."""
    size = L.qar_kv8_attention_shared_workspace_bytes
    for dim in (64, 128, 256):
        queries = (1 << 34) // dim // (64 * 64)
        assert size(64, queries, 64, 8, dim, 4, 1) == size(64, queries, 64, 8, dim, 4, 64) == 0
        assert size(64, queries // 2, 64, 8, dim, 4, 1) > 0
        far = dict(k=1 << 50, v=1 << 51, k_scales=1 << 52, v_scales=1 << 53, page_table=1 << 54, lengths=1 << 55)
        c = ctypes.byref(_struct(**far, batch=64, kv_heads=8, dim=dim))
        assert L.qar_kv8_attention_shared(c, 1 << 40, 0, queries, 64, 600 * M, 610 * M, 1, None, 1.0, 1 << 41, 1 << 42, (1 << 42) - 1,
                                          None) == INV
