"""The serving calls around forked sequences without a GPU: every refusal of the C ABI and of the binding (each call below
fails a check or has nothing to do, so nothing is launched)."""
import ctypes

import pytest
import torch
from test_serve_abi import BAD_CACHES, INV, M, MIS, OK, UNS, _AsCuda, _cache, _struct, _t

from block_wise_int8_amd import qar

I32, BF = torch.int32, torch.bfloat16
REFS, NEW = 2000 * M, dict(page_table=1400 * M, lengths=1500 * M)


@pytest.fixture(scope="module")
def L():
    return qar.lib()


def _calls(L):
    def fork(c, into=None, **kw):
        good = dict(refs=REFS, parents=600 * M, into=into or ctypes.byref(_struct(**NEW)))
        return L.qar_kv8_fork(c, *{**good, **kw}.values(), None)

    def free(c, **kw):
        return L.qar_kv8_free(c, *{**dict(refs=REFS, keep=600 * M), **kw}.values(), None)

    def reserve(c, **kw):
        good = dict(refs=REFS, tokens=600 * M, room=700 * M, source=800 * M, target=900 * M)
        return L.qar_kv8_reserve(c, *{**good, **kw}.values(), None)

    def compact(c, **kw):
        return L.qar_kv8_compact(c, *{**dict(refs=REFS, source=800 * M, target=900 * M), **kw}.values(), None)

    def copy(c, into=None, **kw):
        good = dict(into=into or ctypes.byref(_struct()), source=800 * M, target=900 * M, count=5)
        return L.qar_kv8_copy(c, *{**good, **kw}.values(), None)
    return fork, free, reserve, compact, copy


def test_bad_caches(L):
    for kw, status in BAD_CACHES:
        c = ctypes.byref(_struct(**kw))
        for call in _calls(L):
            assert call(c) == status, (kw, call.__name__)
        fork, copy = _calls(L)[0], _calls(L)[4]
        assert fork(ctypes.byref(_struct()), ctypes.byref(_struct(**{**NEW, **kw}))) == status, kw
        assert copy(ctypes.byref(_struct()), c) == status, kw
    for call in _calls(L):
        assert call(None) == INV


def test_refs(L):
    c = ctypes.byref(_struct())
    for call in _calls(L)[:4]:
        assert call(c, refs=None) == INV and call(c, refs=REFS + 2) == MIS
        for at in (M, 100 * M, 200 * M, 300 * M, 400 * M, 500 * M + 8):
            assert call(c, refs=at) == INV, (call.__name__, at)
        assert call(ctypes.byref(_struct(lengths=400 * M + 44))) == INV                  # the table's last entry
        assert call(ctypes.byref(_struct(batch=1 << 20, table_width=1 << 12))) == INV


def test_fork_refusals(L):
    fork = _calls(L)[0]
    c = ctypes.byref(_struct())
    assert fork(c, ctypes.byref(_struct(**NEW, batch=0))) == OK
    assert fork(c, parents=None) == INV and fork(c, parents=600 * M + 1) == MIS
    for at in (REFS + 36, 1400 * M, 1500 * M, M):
        assert fork(c, parents=at) == INV, at
    for kw in (dict(pages=9), dict(kv_heads=1), dict(dim=128), dict(k=M + 16), dict(v=201 * M), dict(k_scales=101 * M),
               dict(v_scales=301 * M), dict(table_width=3), dict(page_table=400 * M), dict(lengths=500 * M),
               dict(page_table=500 * M), dict(lengths=400 * M)):
        assert fork(c, ctypes.byref(_struct(**{**NEW, **kw}))) == INV, kw


def test_free_and_reserve_and_compact_refusals(L):
    _, free, reserve, compact, _ = _calls(L)
    c = ctypes.byref(_struct())
    for call in (free, reserve):
        assert call(ctypes.byref(_struct(batch=0))) == OK
    assert compact(ctypes.byref(_struct(batch=0))) == INV                                # its lists would stay unset
    assert free(c, keep=600 * M + 2) == MIS and free(c, keep=REFS) == INV and free(c, keep=500 * M + 4) == INV
    for name in ("tokens", "room", "source", "target"):
        assert reserve(c, **{name: None}) == INV and reserve(c, **{name: 1000 * M + 2}) == MIS, name
        for at in (REFS, 400 * M, 500 * M, 200 * M):
            assert reserve(c, **{name: at}) == INV, name
    assert reserve(c, room=600 * M + 8) == INV and reserve(c, source=700 * M) == INV and reserve(c, target=800 * M) == INV
    assert reserve(ctypes.byref(_struct(batch=qar.QAR_KV8_MAX_SEQUENCES + 1))) == INV
    for name in ("source", "target"):
        assert compact(c, **{name: None}) == INV and compact(c, **{name: 1000 * M + 2}) == MIS, name
        for at in (REFS + 36, 400 * M, M):
            assert compact(c, **{name: at}) == INV, name
    assert compact(c, source=900 * M + 16) == INV
    assert compact(ctypes.byref(_struct(pages=1))) == OK                                 # nothing can move


def test_copy_refusals(L):
    copy = _calls(L)[4]
    c = ctypes.byref(_struct())
    assert copy(c, count=0) == OK and copy(c, count=(1 << 30) + 1) == INV
    for name in ("source", "target"):
        assert copy(c, **{name: None}) == INV and copy(c, **{name: 1000 * M + 2}) == MIS and copy(c, **{name: M}) == INV, name
    assert copy(c, source=900 * M + 16) == INV
    for kw in (dict(kv_heads=1), dict(dim=128), dict(k=M + 4096), dict(v=M), dict(k_scales=300 * M), dict(pages=9)):
        assert copy(c, ctypes.byref(_struct(**kw))) == INV, kw
    far = dict(k=1001 * M, k_scales=1100 * M, v=1001 * M + 4096, v_scales=1300 * M)
    assert copy(c, ctypes.byref(_struct(**far))) == INV                                  # keys over values
    many = dict(kv_heads=1 << 20, dim=64)
    assert copy(ctypes.byref(_struct(**many, pages=1)), ctypes.byref(_struct(**many, pages=1))) == INV


def test_norm_rotate_refusals(L):
    good = dict(x=M, dtype=0, batch=2, tokens=3, heads=4, kv_heads=2, dim=64, positions=100 * M, frequencies=200 * M, pairs=32,
                q_gain=300 * M, k_gain=400 * M, eps=1e-6, flags=qar.QAR_ROTATE_NORM, q=500 * M, k=600 * M, v=700 * M)

    def call(**kw):
        return L.qar_norm_rotate(*{**good, **kw}.values(), None)
    assert call(batch=0) == OK and call(tokens=0) == OK
    assert call(dim=96) == UNS and call(dtype=2) == UNS
    assert call(flags=8) == INV and call(flags=0) == INV                                 # gains without a norm
    assert call(heads=0) == INV and call(kv_heads=0) == INV and call(pairs=33) == INV
    assert call(heads=(1 << 20) + 1) == INV and call(kv_heads=(1 << 20) + 1) == INV
    for name in ("x", "positions", "frequencies", "q", "k", "v"):
        assert call(**{name: None}) == INV, name
    for name in ("x", "q_gain", "k_gain", "q", "k", "v"):
        assert call(**{name: 900 * M + 8}) == MIS, name
    assert call(positions=100 * M + 2) == MIS and call(frequencies=200 * M + 1) == MIS
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == INV
    assert call(batch=1 << 40) == INV and call(batch=1 << 20, tokens=1 << 11) == INV and call(tokens=1 << 60) == INV
    assert call(batch=1 << 16, tokens=1 << 13, heads=1 << 20) == INV
    for name in ("q", "k", "v"):
        for at in (M, 100 * M, 200 * M + 112, 300 * M, 400 * M + 112):
            assert call(**{name: at}) == INV, (name, at)
    assert call(q=600 * M) == INV and call(k=700 * M + 16) == INV
    # what is read over positions: eight bytes, or twenty-four
    assert call(q=100 * M + 16, flags=5) == INV


# ---------------------------------------------------------------------------
# the binding


def test_calls_that_do_not_fit():
    c, refs = _cache(), _t(6, dtype=I32)
    three, cpu = _t(3, dtype=I32), torch.zeros(3, dtype=I32)
    x, pos = _t(3, 5, 8, 64), three
    cases = [
        (lambda: qar.qar_kv8_fork(c, _t(5, dtype=I32), three, c.forked(3)), ValueError, "refs must be"),
        (lambda: qar.qar_kv8_fork(c, _t(6), three, c.forked(3)), TypeError, "refs must be torch.int32"),
        (lambda: qar.qar_kv8_fork(c, refs, _t(4, dtype=I32), c.forked(3)), ValueError, "parents must be"),
        (lambda: qar.qar_kv8_fork(c, refs, three, _cache(lengths=_t(4, dtype=I32))), ValueError, "into.lengths must hold 3"),
        (lambda: qar.qar_kv8_fork(c, refs, cpu, c.forked(3)), TypeError, "parents must be a CUDA"),
        (lambda: qar.qar_kv8_free(c, refs, _t(2, dtype=I32)), ValueError, "keep must be"),
        (lambda: qar.qar_kv8_reserve(c, refs, _t(3)), TypeError, "tokens must be torch.int32"),
        (lambda: qar.qar_kv8_reserve(c, refs, three, target=_t(4, dtype=I32)), ValueError, "target must be"),
        (lambda: qar.qar_kv8_compact(c, refs, source=_t(4, dtype=I32)), ValueError, "source must be"),
        (lambda: qar.qar_kv8_copy(c, _t(3, 1, dtype=I32), three), ValueError, "source must have 1 dimension"),
        (lambda: qar.qar_kv8_copy(c, three, _t(4, dtype=I32)), ValueError, "target must be"),
        (lambda: qar.qar_kv8_copy(c, three, _t(3, dtype=torch.int64)), TypeError, "target must be torch.int32"),
        (lambda: qar.qar_kv8_copy(c, three, three, into=_cache(k=None)), TypeError, "into.k must be a CUDA"),
        (lambda: qar.qar_norm_rotate(x, 4, 1, pos), ValueError, "qkv must be"),
        (lambda: qar.qar_norm_rotate(x, True, 2, pos), ValueError, "heads must be a whole number"),
        (lambda: qar.qar_norm_rotate(x, 8, 0, pos), ValueError, "kv_heads must be a whole number"),
        (lambda: qar.qar_norm_rotate(x[0], 4, 2, pos), ValueError, "qkv must be"),
        (lambda: qar.qar_norm_rotate(x.half().as_subclass(_AsCuda), 4, 2, pos), TypeError, "bfloat16 and float32"),
        (lambda: qar.qar_norm_rotate(x, 4, 2, _t(3, 4, dtype=I32)), ValueError, "positions must be"),
        (lambda: qar.qar_norm_rotate(x, 4, 2, _t(3, dtype=torch.int64)), TypeError, "positions must be torch.int32"),
        (lambda: qar.qar_norm_rotate(x, 4, 2, pos, _t(32, dtype=torch.float64)), TypeError, "frequencies must be"),
        (lambda: qar.qar_norm_rotate(x, 4, 2, pos, _t(1, 32)), ValueError, "frequencies must have 1"),
        (lambda: qar.qar_norm_rotate(x, 4, 2, pos, q_gain=_t(64, dtype=BF), eps=0.1), TypeError, "q_gain must be"),
        (lambda: qar.qar_norm_rotate(x, 4, 2, pos, k_gain=_t(63), eps=0.1), ValueError, "k_gain must be"),
        (lambda: qar.qar_norm_rotate(x, 4, 2, pos, interleaved=1), TypeError, "interleaved must be"),
        (lambda: qar.qar_norm_rotate(x, 4, 2, pos, out=(x, x)), ValueError, "out must be"),
        (lambda: qar.qar_norm_rotate(x, 4, 2, pos, out=(x, x, x)), ValueError, "out.0. must be"),
    ]
    for i, (call, error, text) in enumerate(cases):
        with pytest.raises(error, match=text):
            call()
            pytest.fail(f"case {i} was not refused")


def test_the_extension_counts_arguments_and_hands_back():
    ext = qar._serve()
    for name, count in (("kv8_fork", 4), ("kv8_free", 3), ("kv8_reserve", 6), ("kv8_compact", 4), ("kv8_copy", 4),
                        ("norm_rotate", 10)):
        for wrong in (0, count - 1, count + 1):
            with pytest.raises(TypeError, match=f"{count} arguments"):
                getattr(ext, name)(*[None] * wrong)
        assert getattr(ext, name)(*[None] * count) is None
    c = qar.KvCache.empty(4, 2, 64, 2, 2, device="cpu")
    assert ext.kv8_free(c, torch.zeros(4, dtype=I32), None) is None


def test_forked_tables():
    c = qar.KvCache.empty(4, 2, 64, 2, 3, device="cpu")
    f = c.forked(5)
    assert f.k is c.k and f.v_scales is c.v_scales and f.page_table.shape == (5, 3) and f.lengths.shape == (5,)
    assert c.forked(1, 9).page_table.shape == (1, 9) and f.page_table.dtype == I32


# ---------------------------------------------------------------------------
# the product with an epilogue


def test_mx4_linear_fused_refusals(L):
    good = dict(x=M, dtype=0, rows=4, inner=96, codes=2 * M, scales=3 * M, cols=50, bias=5 * M, activation=1, residual=6 * M,
                out=4 * M, out_dtype=0, ws=None, size=0)

    def call(**kw):
        return L.qar_mx4_linear_fused(*{**good, **kw}.values(), None)
    assert call(rows=0) == OK and call(cols=0) == OK and call(inner=0) == INV
    for name in ("x", "codes", "scales", "out"):
        assert call(**{name: None}) == INV, name
    assert call(dtype=2) == UNS and call(out_dtype=7) == UNS and call(activation=5) == UNS and call(activation=-1) == UNS
    for name in ("x", "codes", "bias", "residual", "out"):
        assert call(**{name: 7 * M + 8}) == MIS, name
    assert call(out=2 * M) == INV and call(out=5 * M + 80) == INV and call(bias=4 * M + 384) == INV
    assert call(residual=4 * M + 16) == INV and call(residual=4 * M - 16) == INV         # the output only as a whole
    need = L.qar_mx4_linear_workspace_bytes(40, 96, 50)
    assert call(rows=40) == INV and call(rows=40, ws=8 * M, size=need - 1) == INV
    for at in (4 * M, 5 * M, 6 * M, M):
        assert call(rows=40, ws=at, size=need) == INV
    assert call(rows=1 << 21, inner=1 << 20) == INV


def test_mx4_linear_fused_arguments():
    u8 = torch.uint8
    x, codes, scales = _t(2, 32), _t(5, 16, dtype=u8), _t(5, 1, dtype=u8)
    cases = [
        (dict(bias=_t(4)), ValueError, "bias must be"), (dict(bias=_t(5, dtype=BF)), TypeError, "bias must be torch.float32"),
        (dict(bias=_t(5), out_dtype=BF), TypeError, "bias must be torch.bfloat16"),
        (dict(residual=_t(2, 4)), ValueError, "residual must hold 10"),
        (dict(residual=_t(2, 5), out=_t(2, 5, dtype=BF)), TypeError, "residual must be torch.bfloat16"),
        (dict(activation="tanh"), ValueError, "activation must be"), (dict(activation=1), ValueError, "activation must be"),
        (dict(out=_t(2, 4)), ValueError, "out must hold 10"), (dict(out_dtype=torch.float16), TypeError, "bfloat16 and float32")]
    for i, (kw, error, text) in enumerate(cases):
        with pytest.raises(error, match=text):
            qar.qar_mx4_linear_fused(x, codes, scales, **kw)
            pytest.fail(f"case {i} was not refused")
    ext = qar._serve()
    assert ext.mx4_linear_fused(*[None] * 9) is None
    with pytest.raises(TypeError, match="9 arguments"):
        ext.mx4_linear_fused(None)


# ---------------------------------------------------------------------------
# attention behind shared prefixes


def test_attention_shared_refusals(L):
    size = L.qar_kv8_attention_shared_workspace_bytes
    need = size(3, 1, 4, 2, 64, 4, 2)
    assert need > 0 and need % 256 == 0
    good = dict(q=600 * M, dtype=0, queries=1, heads=4, starts=610 * M, prefix=620 * M, groups=2, q_lens=None, scale=1.0,
                out=700 * M, ws=800 * M, size=need)

    def call(c=None, **kw):
        return L.qar_kv8_attention_shared(c or ctypes.byref(_struct()), *{**good, **kw}.values(), None)
    assert call(queries=0) == OK and call(ctypes.byref(_struct(batch=0))) == OK
    for kw, status in BAD_CACHES:
        assert call(ctypes.byref(_struct(**kw))) == status, kw
    for name in ("q", "out", "starts", "prefix", "ws"):
        assert call(**{name: None}) == INV, name
    assert call(groups=0) == INV and call(groups=4) == INV and call(heads=3) == INV and call(heads=0) == INV
    assert call(queries=(1 << 30) + 1) == INV and call(dtype=2) == UNS
    assert call(q=600 * M + 8) == MIS and call(out=700 * M + 8) == MIS and call(q_lens=900 * M + 2) == MIS
    assert call(starts=610 * M + 2) == MIS and call(prefix=620 * M + 1) == MIS and call(ws=800 * M + 128) == MIS
    assert call(size=need - 1) == INV
    for at in (600 * M, 610 * M, 620 * M, 200 * M, 500 * M, 800 * M):
        assert call(out=at) == INV, at
    for at in (600 * M, 610 * M, 620 * M, M, 700 * M):
        assert call(ws=at) == INV, at
    assert call(q_lens=700 * M) == INV and call(out=610 * M - 16) == INV
    assert size(0, 1, 4, 2, 64, 4, 1) == size(3, 0, 4, 2, 64, 4, 1) == size(3, 1, 3, 2, 64, 4, 1) == size(3, 1, 4, 2, 80, 4, 1) == 0
    assert size(3, 1, 4, 2, 64, 0, 1) == size(3, 1, 4, 2, 64, 4, 0) == size(3, 1, 4, 2, 64, 4, 4) == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_shared_workspace(L, dim):
    """A slot of the prefix and one of the own pages at least: a maximum, a sum and a row of outputs for each row."""
    for batch, queries, heads, kv_heads, width, groups in [(1, 1, 1, 1, 1, 1), (64, 1, 32, 8, 600, 1), (64, 1, 32, 8, 600, 64),
                                                           (3, 500, 12, 12, 40, 2), (1000, 1, 8, 1, 9, 7)]:
        assert L.qar_kv8_attention_shared_workspace_bytes(batch, queries, heads, kv_heads, dim, width, groups) >= \
            batch * queries * heads * 2 * (dim * 4 + 8)


def test_attention_shared_arguments():
    c, q, three, one = _cache(), _t(3, 1, 4, 64), _t(3, dtype=I32), _t(1, dtype=I32)
    two = _t(2, dtype=I32)
    cases = [(dict(starts=one, prefix=one), ValueError, "starts must be"), (dict(starts=three, prefix=three), ValueError, "prefix must be"),
             (dict(starts=_t(2), prefix=one), TypeError, "starts must be torch.int32"), (dict(starts=two, prefix=_t(1)), TypeError, "prefix"),
             (dict(q=_t(3, 4, 64)), ValueError, "q must be"), (dict(q_lens=two), ValueError, "q_lens must be"),
             (dict(out=_t(3, 1, 4, 32)), ValueError, "out must be"), (dict(workspace=torch.zeros(3)), TypeError, "workspace must be")]
    for i, (kw, error, text) in enumerate(cases):
        with pytest.raises(error, match=text):
            qar.qar_kv8_attention_shared(c, **{**dict(q=q, starts=two, prefix=one), **kw})
            pytest.fail(f"case {i} was not refused")
    assert qar._serve().kv8_attention_shared(*[None] * 8) is None


def test_the_header_beside_the_kernels_holds_no_vector_assembly():
    """What tests/test_serve_sources.py asks of the kernels' sources, of the header that they share."""
    import os
    import re

    from block_wise_int8_amd import build
    text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, "qar_kv8_device.h")).read())
    for s in re.findall(r"\basm\b[^;]*;", text):
        assert not re.search(r'"[^"]*\bv_\w+', s), s
