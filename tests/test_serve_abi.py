"""The serving calls without a GPU: every refusal of the C ABI and of the
binding (each call below fails a check, so nothing is launched), and the
workspace sizes."""
import ctypes

import numpy as np
import pytest
import serve_reference as ref
import torch

from block_wise_int8_amd import qar

INV, MIS, UNS, OK = qar.QAR_ERR_INVALID_ARG, qar.QAR_ERR_MISALIGNED, qar.QAR_ERR_UNSUPPORTED, qar.QAR_OK
M = 1 << 20                       # fake, aligned device addresses (never dereferenced), a MiB apart or more


@pytest.fixture(scope="module")
def L():
    return qar.lib()


# ---------------------------------------------------------------------------
# 4-bit


def test_mx4_quantize_refusals(L):
    q = L.qar_mx4_quantize
    good = dict(x=M, dtype=0, rows=4, cols=100, codes=2 * M, scales=3 * M)

    def call(**kw):
        return q(*{**good, **kw}.values(), None)
    assert call(rows=0) == OK and call(cols=0) == OK
    for name in ("x", "codes", "scales"):
        assert call(**{name: None}) == INV, name
    assert call(dtype=2) == UNS and call(dtype=-1) == UNS
    assert call(x=M + 8) == MIS and call(codes=2 * M + 4) == MIS
    assert call(rows=(1 << 30) + 1) == INV and call(cols=(1 << 30) + 1) == INV
    assert call(rows=1 << 30, cols=1 << 30) == INV
    assert call(codes=M + 4 * 100 * 2 - 16) == INV                   # the last bytes of x
    assert call(scales=2 * M + 4 * 4 * 16 - 1) == INV                # of the codes (4 blocks a row)
    assert call(scales=M + 1) == INV


def test_mx4_dequantize_refusals(L):
    d = L.qar_mx4_dequantize
    good = dict(codes=M, scales=2 * M, rows=4, cols=100, out=3 * M, dtype=1)

    def call(**kw):
        return d(*{**good, **kw}.values(), None)
    assert call(rows=0) == OK and call(cols=0) == OK
    for name in ("codes", "scales", "out"):
        assert call(**{name: None}) == INV, name
    assert call(dtype=2) == UNS
    assert call(codes=M + 8) == MIS and call(out=3 * M + 2) == MIS
    assert call(cols=(1 << 30) + 1) == INV
    assert call(out=M + 240) == INV and call(scales=3 * M + 1599) == INV


def test_mx4_linear_refusals(L):
    f = L.qar_mx4_linear
    good = dict(x=M, dtype=0, rows=4, inner=96, codes=2 * M, scales=3 * M, cols=50, out=4 * M, out_dtype=0, ws=None, size=0)

    def call(**kw):
        return f(*{**good, **kw}.values(), None)
    assert call(rows=0) == OK and call(cols=0) == OK and call(inner=0) == INV
    for name in ("x", "codes", "scales", "out"):
        assert call(**{name: None}) == INV, name
    assert call(dtype=2) == UNS and call(out_dtype=7) == UNS
    assert call(x=M + 2) == MIS and call(codes=2 * M + 8) == MIS and call(out=4 * M + 4) == MIS
    assert call(out=M + 752) == INV and call(out=2 * M) == INV and call(scales=4 * M + 399) == INV
    need = L.qar_mx4_linear_workspace_bytes(40, 96, 50)
    assert need > 0
    assert call(rows=40) == INV                                      # no workspace
    assert call(rows=40, ws=8 * M, size=need - 1) == INV
    assert call(rows=40, ws=8 * M + 64, size=need) == MIS
    assert call(rows=40, ws=4 * M + 256, size=need) == INV           # over the output
    assert call(rows=40, ws=2 * M, size=need) == INV
    for big in (dict(rows=(1 << 30) + 1), dict(inner=(1 << 30) + 1), dict(cols=(1 << 30) + 1),
                dict(rows=1 << 21, inner=1 << 20), dict(cols=1 << 21, inner=1 << 20), dict(rows=1 << 21, cols=1 << 20)):
        assert call(**big) == INV, big


def test_mx4_linear_workspace(L):
    size = L.qar_mx4_linear_workspace_bytes
    assert size(0, 1, 1) == size(1, 0, 1) == size(1, 1, 0) == 0
    assert size(16, 4992, 5000) == 0                                 # few rows of whole blocks are quantized in registers
    for rows in (1, 17, 64, 65, 1000):
        assert size(rows, 1000, 300) >= rows * 32 * 17               # the codes and scales of x
        assert size(rows, 1000, 300) % 256 == 0
    assert size(1 << 31, 64, 64) == 0


# ---------------------------------------------------------------------------
# the cache


class _Kv(ctypes.Structure):
    """qar_kv8_cache"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "k_scales", "v", "v_scales", "page_table", "lengths")] + \
        [(n, ctypes.c_uint32) for n in ("pages", "kv_heads", "dim", "batch", "table_width")]


def test_the_binding_packs_the_struct():
    c = _Kv(*[i << 40 for i in range(1, 7)], 7, 8, 9, 10, 11)
    assert bytes(c) == qar._KV_PACK(*[i << 40 for i in range(1, 7)], 7, 8, 9, 10, 11)


def _struct(**kw):
    good = dict(k=M, k_scales=100 * M, v=200 * M, v_scales=300 * M, page_table=400 * M, lengths=500 * M, pages=10,
                kv_heads=2, dim=64, batch=3, table_width=4)
    return _Kv(*{**good, **kw}.values())


BAD_CACHES = [(dict(dim=96), UNS), (dict(dim=0), UNS), (dict(k=None), INV), (dict(k_scales=None), INV), (dict(v=None), INV),
              (dict(v_scales=None), INV), (dict(page_table=None), INV), (dict(lengths=None), INV), (dict(pages=0), INV),
              (dict(pages=1 << 31), INV), (dict(kv_heads=0), INV), (dict(table_width=0), INV),
              (dict(table_width=(1 << 24) + 1), INV), (dict(pages=(1 << 31) - 1, kv_heads=1 << 10), INV),
              (dict(k=M + 8), MIS), (dict(v=200 * M + 4), MIS), (dict(k_scales=100 * M + 2), MIS),
              (dict(v_scales=300 * M + 1), MIS), (dict(page_table=400 * M + 2), MIS), (dict(lengths=500 * M + 3), MIS)]


def _calls(L):
    def append(c, **kw):
        good = dict(starts=600 * M, k=700 * M, v=800 * M, dtype=0, tokens=5)
        return L.qar_kv8_append(c, *{**good, **kw}.values(), None)

    def read(c, **kw):
        good = dict(starts=600 * M, tokens=5, k=700 * M, v=800 * M, dtype=0)
        return L.qar_kv8_read(c, *{**good, **kw}.values(), None)

    def attend(c, **kw):
        good = dict(q=600 * M, dtype=0, queries=1, heads=4, q_lens=None, scale=1.0, weights=None, out=700 * M, ws=None, size=0)
        return L.qar_kv8_attention(c, *{**good, **kw}.values(), None)

    def evict(c, into=None, **kw):
        other = _struct(k=1001 * M, k_scales=1100 * M, v=1200 * M, v_scales=1300 * M, page_table=1400 * M, lengths=1500 * M)
        good = dict(weights=600 * M, recent=5, keep=100, kept=700 * M, moved=800 * M)
        return L.qar_kv8_evict(c, into or ctypes.byref(other), *{**good, **kw}.values(), None)
    return append, read, attend, evict


def test_bad_caches(L):
    for kw, status in BAD_CACHES:
        c = ctypes.byref(_struct(**kw))
        for call in _calls(L):
            assert call(c) == status, (kw, call.__name__)
        assert _calls(L)[3](ctypes.byref(_struct()), c) == status, kw
    for call in _calls(L):
        assert call(None) == INV


def test_append_refusals(L):
    append = _calls(L)[0]
    c = ctypes.byref(_struct())
    assert append(c, tokens=0) == OK and append(ctypes.byref(_struct(batch=0))) == OK
    for name in ("starts", "k", "v"):
        assert append(c, **{name: None}) == INV, name
    assert append(c, dtype=3) == UNS
    assert append(c, starts=600 * M + 2) == MIS and append(c, k=700 * M + 8) == MIS and append(c, v=800 * M + 2) == MIS
    assert append(c, k=M) == INV and append(c, v=200 * M) == INV and append(c, starts=300 * M) == INV
    assert append(c, tokens=(1 << 30) + 1) == INV
    assert append(ctypes.byref(_struct(batch=1 << 20, kv_heads=64)), tokens=64 * 1000) == INV      # too many workgroups
    assert append(ctypes.byref(_struct(v=M))) == INV and append(ctypes.byref(_struct(page_table=M + 64))) == INV


def test_read_refusals(L):
    read = _calls(L)[1]
    c = ctypes.byref(_struct())
    assert read(c, tokens=0) == OK
    for name in ("starts", "k", "v"):
        assert read(c, **{name: None}) == INV, name
    assert read(c, dtype=3) == UNS
    assert read(c, starts=600 * M + 2) == MIS and read(c, k=700 * M + 8) == MIS and read(c, v=800 * M + 2) == MIS
    assert read(c, k=800 * M) == INV and read(c, k=200 * M) == INV and read(c, v=500 * M) == INV and read(c, k=600 * M) == INV
    assert read(c, tokens=(1 << 30) + 1) == INV


def test_attention_refusals(L):
    attend = _calls(L)[2]
    c = ctypes.byref(_struct())
    assert attend(c, queries=0) == OK
    assert attend(c, q=None) == INV and attend(c, out=None) == INV
    assert attend(c, heads=3) == INV and attend(c, heads=0) == INV and attend(c, queries=(1 << 30) + 1) == INV
    assert attend(c, dtype=2) == UNS
    assert attend(c, q=600 * M + 8) == MIS and attend(c, out=700 * M + 8) == MIS and attend(c, q_lens=900 * M + 2) == MIS
    assert attend(c, weights=900 * M + 1) == MIS
    assert attend(c, out=600 * M) == INV and attend(c, out=200 * M) == INV and attend(c, q_lens=700 * M) == INV
    size = L.qar_kv8_attention_workspace_bytes
    need = size(3, 1, 4, 2, 64, 4, 0, 1)
    assert need > 0
    assert attend(c, weights=900 * M) == INV                                             # no workspace
    assert attend(c, weights=900 * M, ws=950 * M, size=need - 1) == INV
    assert attend(c, weights=900 * M, ws=950 * M + 128, size=need) == MIS
    assert attend(c, weights=900 * M, ws=900 * M, size=need) == INV                      # over the weights
    assert attend(c, weights=700 * M, ws=950 * M, size=need) == INV                      # over the output
    assert attend(c, weights=M, ws=950 * M, size=need) == INV
    assert size(0, 1, 4, 2, 64, 4, 0, 1) == size(3, 1, 3, 2, 64, 4, 0, 1) == size(3, 1, 4, 2, 80, 4, 0, 1) == 0
    assert size(3, 1, 4, 2, 64, 4, 2, 1) == 0 and size(3, 40, 4, 2, 64, 4, 1, 1) > size(3, 40, 4, 2, 64, 4, 0, 1)


def test_evict_refusals(L):
    evict = _calls(L)[3]
    c = ctypes.byref(_struct())
    for name in ("weights", "kept", "moved"):
        assert evict(c, **{name: None}) == INV, name
    assert evict(c, keep=0) == INV and evict(c, keep=257) == INV                         # into's table has 4 pages
    assert evict(c, kept=700 * M + 2) == MIS and evict(c, moved=800 * M + 1) == MIS and evict(c, weights=600 * M + 2) == MIS
    assert evict(c, kept=800 * M) == INV and evict(c, moved=600 * M) == INV and evict(c, kept=M) == INV
    assert evict(c, kept=1001 * M) == INV
    far = dict(k=1001 * M, k_scales=1100 * M, v=1200 * M, v_scales=1300 * M, page_table=1400 * M, lengths=1500 * M)
    for kw in (dict(batch=4), dict(kv_heads=1), dict(dim=128), dict(lengths=500 * M), dict(k=M + 16), dict(k_scales=200 * M),
               dict(lengths=600 * M), dict(v=1001 * M)):
        assert evict(c, ctypes.byref(_struct(**{**far, **kw}))) == INV, kw


# ---------------------------------------------------------------------------
# the binding


class _AsCuda(torch.Tensor):
    """A host tensor that reports itself as a device tensor, so that the checks behind that one refuse it."""
    @property
    def is_cuda(self):
        return True


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_AsCuda)


def _cache(**kw):
    c = dict(k=_t(6, 2, 64, 64, dtype=torch.int8), k_scales=_t(6, 2), v=_t(6, 2, 64, 64, dtype=torch.int8),
             v_scales=_t(6, 2), page_table=_t(3, 2, dtype=torch.int32), lengths=_t(3, dtype=torch.int32))
    return qar.KvCache(**{**c, **kw})


STARTS = _t(3, dtype=torch.int32)


def test_host_tensors_are_refused():
    with pytest.raises(TypeError, match="CUDA"):
        qar.qar_mx4_quantize(torch.zeros(2, 32))
    with pytest.raises(TypeError, match="CUDA"):
        qar.qar_kv8_read(qar.KvCache.empty(2, 1, 64, 1, 1, device="cpu"), STARTS, 1)


@pytest.mark.parametrize("kw,error,text", [
    (dict(k=_t(6, 2, 32, 64, dtype=torch.int8)), ValueError, "cache.k must be"),
    (dict(k=_t(6, 2, 64, 64)), TypeError, "cache.k must be torch.int8"),
    (dict(v=_t(6, 2, 64, 128, dtype=torch.int8)), ValueError, "cache.v must be"),
    (dict(v=_t(6, 2, 64, 64, dtype=torch.uint8)), TypeError, "cache.v must be torch.int8"),
    (dict(k_scales=_t(6)), ValueError, "cache.k_scales must hold 12"),
    (dict(v_scales=_t(6, 2, dtype=torch.bfloat16)), TypeError, "cache.v_scales must be torch.float32"),
    (dict(page_table=_t(3, 2, dtype=torch.int64)), TypeError, "cache.page_table must be torch.int32"),
    (dict(page_table=_t(6, dtype=torch.int32)), ValueError, "page_table"),
    (dict(lengths=_t(2, dtype=torch.int32)), ValueError, "cache.lengths must hold 3"),
    (dict(k_scales=_t(2, 6).t()), ValueError, "cache.k_scales must be contiguous")])
def test_caches_that_do_not_fit(kw, error, text):
    with pytest.raises(error, match=text):
        qar.qar_kv8_read(_cache(**kw), STARTS, 1)


def test_calls_that_do_not_fit():
    c, bf = _cache(), torch.bfloat16
    cases = [
        (lambda: qar.qar_kv8_append(c, STARTS, _t(3, 1, 2, 32), _t(3, 1, 2, 32)), ValueError, "k_new must be"),
        (lambda: qar.qar_kv8_append(c, STARTS, _t(3, 2, 64), _t(3, 2, 64)), ValueError, "k_new must be"),
        (lambda: qar.qar_kv8_append(c, STARTS, _t(3, 1, 2, 64), _t(3, 2, 2, 64)), ValueError, "v_new must be"),
        (lambda: qar.qar_kv8_append(c, STARTS, _t(3, 1, 2, 64), _t(3, 1, 2, 64, dtype=bf)), TypeError, "v_new must be"),
        (lambda: qar.qar_kv8_append(c, _t(3), _t(3, 1, 2, 64), _t(3, 1, 2, 64)), TypeError, "starts must be torch.int32"),
        (lambda: qar.qar_kv8_read(c, _t(2, dtype=torch.int32), 1), ValueError, "starts must be"),
        (lambda: qar.qar_kv8_read(c, STARTS, 1, out=(_t(3, 1, 2, 64), _t(3, 1, 2, 63))), ValueError, "out.1. must be"),
        (lambda: qar.qar_kv8_attention(c, _t(3, 4, 64)), ValueError, "q must be"),
        (lambda: qar.qar_kv8_attention(c, _t(3, 1, 4, 64, dtype=torch.float16)), TypeError, "q must be"),
        (lambda: qar.qar_kv8_attention(c, _t(3, 1, 4, 64), q_lens=_t(3)), TypeError, "q_lens must be"),
        (lambda: qar.qar_kv8_attention(c, _t(3, 1, 4, 64), weights=_t(3, 2, 64)), ValueError, "weights must be"),
        (lambda: qar.qar_kv8_attention(c, _t(3, 1, 4, 64), out=_t(3, 1, 4, 64, dtype=bf)), TypeError, "out must be"),
        (lambda: qar.qar_kv8_evict(c, _cache(), _t(3, 2, 127), 1, 1), ValueError, "weights must be"),
        (lambda: qar.qar_kv8_evict(c, _cache(), _t(3, 2, 128), -1, 1), ValueError, "recent must be"),
        (lambda: qar.qar_kv8_evict(c, _cache(), _t(3, 2, 128), 1, 0), ValueError, "keep at least 1"),
        (lambda: qar.qar_kv8_evict(c, _cache(), _t(3, 2, 128), 1, 5, kept=_t(3, 2, 5)), TypeError, "kept must be"),
        (lambda: qar.qar_mx4_quantize(_t(4)), ValueError, "x must have 2 dimensions"),
        (lambda: qar.qar_mx4_quantize(_t(4, 4, dtype=torch.float16)), TypeError, "bfloat16 and float32"),
        (lambda: qar.qar_mx4_quantize(_t(2, 33), codes=_t(2, 16, dtype=torch.uint8)), ValueError, "codes must hold 64"),
        (lambda: qar.qar_mx4_dequantize(_t(2, 16, dtype=torch.uint8), _t(2, 1, dtype=torch.uint8), 33), ValueError, "codes must hold 64"),
        (lambda: qar.qar_mx4_dequantize(_t(2, 16, dtype=torch.uint8), _t(2, 2, dtype=torch.uint8), 32), ValueError, "scales must hold 2"),
        (lambda: qar.qar_mx4_linear(_t(2, 64), _t(5, 16, dtype=torch.uint8), _t(5, 1, dtype=torch.uint8)), ValueError, "codes must hold 160"),
        (lambda: qar.qar_mx4_linear(_t(2, 32), _t(5, 16, dtype=torch.uint8), _t(5, 1, dtype=torch.int8)), TypeError, "scales must be"),
        (lambda: qar.qar_mx4_linear(_t(2, 32), _t(5, 16, dtype=torch.uint8), _t(5, 1, dtype=torch.uint8), out=_t(2, 4)), ValueError, "out must hold 10"),
    ]
    for i, (call, error, text) in enumerate(cases):
        with pytest.raises(error, match=text):
            call()
            pytest.fail(f"case {i} was not refused")


# ---------------------------------------------------------------------------
# the reference that the GPU tests compare with


def test_reference_mx4():
    x = np.zeros((1, 40), np.float32)
    x[0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7]             # midpoints, and a peak in [4, 8): scale 2^0
    x[0, 32:] = -1.0                                                 # peak 1: scale 2^-2, quotient 4
    codes, scales = ref.mx4_quantize(x)
    assert scales.tolist() == [[127, 125]]
    assert codes[0, :4].tolist() == [0x20, 0x42, 0x64, 0x76]
    assert ref.mx4_values(codes, scales, 40)[0, [0, 1, 2, 3, 4, 5, 6, 7, 39]].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, -1]


def test_reference_attention_against_a_loop():
    rng = np.random.default_rng(0)
    c = ref.make_cache(rng, 1, 1, 64, [3], 1)
    q = rng.standard_normal((1, 2, 1, 64)).astype(np.float32)
    r = ref.attend(c, q, [2], 0.125)
    i = c["page_table"][0, 0]
    k = c["k"][i, 0, :3].astype(np.float32) * c["k_scales"][i, 0]
    v = c["v"][i, 0, :, :3].T.astype(np.float32) * c["v_scales"][i, 0]
    for row, sees in ((0, 2), (1, 3)):
        e = [np.exp(0.125 * float(k[t].astype(np.float64) @ q[0, row, 0])) for t in range(sees)]
        want = sum(e[t] * v[t].astype(np.float64) for t in range(sees)) / sum(e)
        assert np.allclose(r["out"][0, row, 0], want, rtol=1e-12)
    assert np.isclose(r["weights"].sum(), 2)
