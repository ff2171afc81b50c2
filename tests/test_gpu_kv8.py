"""The 8-bit paged cache on the GPU against tests/serve_reference.py."""
import numpy as np
import pytest
import serve_reference as ref
import torch

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64
DTYPES = [torch.bfloat16, torch.float32]


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _same_cache(got, want, what, tokens=None):
    """Scales and codes equal; with `tokens`, codes only of each sequence's first tokens[b] tokens and the pages outside the
    table."""
    for name in ("k_scales", "v_scales", "page_table", "lengths"):
        g = getattr(got, name).cpu().numpy()
        assert np.array_equal(g, want[name], equal_nan=g.dtype == np.float32), f"{what}: {name}"
    care = np.ones((want["k"].shape[0], PAGE), bool)
    if tokens is not None:
        for b, n in enumerate(tokens):
            for p in range(want["page_table"].shape[1]):
                i = ref.page_id(want, b, p)
                if i >= 0:
                    care[i] = np.arange(PAGE) + p * PAGE < n
    k, v = got.k.cpu().numpy(), got.v.cpu().numpy()
    assert np.array_equal(k[care.nonzero()[0], :, care.nonzero()[1]],
                          want["k"][care.nonzero()[0], :, care.nonzero()[1]]), f"{what}: key codes"
    assert np.array_equal(v.transpose(0, 3, 1, 2)[care], want["v"].transpose(0, 3, 1, 2)[care]), f"{what}: value codes"


# ---------------------------------------------------------------------------
# append and read


APPENDS = [(1, 1, 1, 64, [0]), (3, 1, 2, 128, [0, 63, 64]), (2, 5, 3, 64, [62, 130]), (2, 64, 1, 256, [0, 1]),
           (1, 200, 2, 128, [37]), (4, 1, 2, 256, [5, 127, 128, 200]), (2, 129, 1, 64, [63, 0]), (3, 7, 2, 128, [-4, 3, 60])]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("grow", [0.01, 1.0, 30.0])
@pytest.mark.parametrize("batch,tokens,heads,dim,starts", APPENDS)
def test_append(batch, tokens, heads, dim, starts, grow, dtype):
    """Bit for bit, with new values far below, around and above what the pages hold."""
    rng = np.random.default_rng(sum(starts) + tokens + dim)
    width = -(-(max(starts) + tokens) // PAGE)
    lengths = [max(0, s + tokens) for s in starts]
    c = ref.make_cache(rng, batch, heads, dim, lengths, width)
    cache = ref.to_cache(c)
    k, kf = ref.data(rng, (batch, tokens, heads, dim), dtype)
    v, vf = ref.data(rng, (batch, tokens, heads, dim), dtype)
    k, v = k * grow, v * grow
    ref.append(c, starts, k.float().cpu().numpy(), v.float().cpu().numpy())
    qar.qar_kv8_append(cache, _ints(*starts), k, v)
    _same_cache(cache, c, "append", lengths)


def test_append_of_zeros_and_extremes():
    rng = np.random.default_rng(3)
    c = ref.make_cache(rng, 2, 1, 64, [70, 70], 2)
    cache = ref.to_cache(c)
    k = torch.zeros((2, 4, 1, 64), device=DEV)
    v = torch.full((2, 4, 1, 64), 3e38, device=DEV)
    k[1] = 1e-44                                                       # subnormal scales
    for starts in ([0, 0], [66, 64]):
        ref.append(c, starts, k.cpu().numpy(), v.cpu().numpy())
        qar.qar_kv8_append(cache, _ints(*starts), k, v)
        _same_cache(cache, c, f"append at {starts}", [70, 70])


def test_append_leaves_out_what_is_not_there():
    """Entries outside the pool, positions behind the table: nothing else changes."""
    rng = np.random.default_rng(4)
    c = ref.make_cache(rng, 3, 2, 64, [190, 190, 190], 3, absent=[(0, 1), (1, 0), (1, 1), (2, 2)])
    cache = ref.to_cache(c)
    k, kf = ref.data(rng, (3, 100, 2, 64), torch.float32)
    ref.append(c, [60, 30, 150], kf, 2 * kf)
    qar.qar_kv8_append(cache, _ints(60, 30, 150), k, 2 * k)
    _same_cache(cache, c, "append", [160, 130, 190])


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("dim,heads,tokens,starts", [(64, 2, 1, [0, 63, 64]), (128, 1, 65, [0, 64, 100]),
                                                     (256, 3, 130, [1, 127, 190]), (64, 1, 300, [-1, 0, 250])])
def test_read(dim, heads, tokens, starts, out):
    rng = np.random.default_rng(tokens + dim)
    lengths = [200, 129, 255]
    c = ref.make_cache(rng, 3, heads, dim, lengths, 4, absent=[(0, 1), (2, 2)])
    got = qar.qar_kv8_read(ref.to_cache(c), _ints(*starts), tokens, out_dtype=out)
    for which, g in zip("kv", got):
        want = np.zeros((3, tokens, heads, dim), np.float32)
        for b in range(3):
            if starts[b] < 0:
                continue
            for h in range(heads):
                x, _ = ref.sequence(c, b, h, which, lengths[b])
                part = x[starts[b]:starts[b] + tokens]
                want[b, :len(part), h] = part
        assert torch.equal(g.cpu(), torch.from_numpy(want).to(out)), which


# ---------------------------------------------------------------------------
# attention


def _attention_tolerance(want, q, dtype, dim, n):
    """What the arithmetic can do to a row: scores are sums of `dim` exact products in binary32 (queries exact in bf16, off
    by 2^-23 of an element in binary32) and a few roundings of numbers no larger than the sum of magnitudes; a numerator
    then is off by that, the exponential's 2^-21 and, entering the product, 2^-12 (one binary16 term) or 2^-22 (two); sums
    over n keys add n 2^-24.  The softmax's sum doubles the scores' part.  Numerators enter the product times 2^14, so those
    below 2^-28 of the row's largest are binary16 subnormals, off by up to 2^-39 each."""
    delta = (dim + 8) * 2.0 ** -23 * want["peak"] + 2.0 ** -20
    rel = 2 * delta + (2.0 ** -12 if dtype == torch.bfloat16 else 2.0 ** -22) + (n + 8) * 2.0 ** -24
    floor = n * 2.0 ** -39 * want["vmax"][..., None] + 1e-37
    return rel[..., None] * want["mass"] + ref.half_step(dtype) * np.abs(want["out"]) + floor, delta


def _check_attention(c, batch, queries, heads, dtype, q_lens=None, weights=False, scale=None, seed=0, spread=1.5):
    rng = np.random.default_rng(seed)
    dim = c["k"].shape[3]
    kv_heads, width = c["k"].shape[1], c["page_table"].shape[1]
    q = (torch.from_numpy(rng.standard_normal((batch, queries, heads, dim)).astype(np.float32)) * spread).to(dtype)
    lens = [queries] * batch if q_lens is None else q_lens
    want = ref.attend(c, q.float().numpy(), lens, dim ** -0.5 if scale is None else scale)
    w0 = rng.uniform(0, 1, (batch, kv_heads, width * PAGE)).astype(np.float32)
    w = _dev(w0) if weights else None
    cache = ref.to_cache(c)
    out = qar.qar_kv8_attention(cache, q.to(DEV), q_lens=None if q_lens is None else _ints(*q_lens), scale=scale, weights=w)
    n = int(max(0, c["lengths"].max()))
    tol, delta = _attention_tolerance(want, q, dtype, dim, n)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - want["out"]) - tol
    assert (over <= 0).all(), (f"{(over > 0).sum()} of {over.size} off, worst at {np.unravel_index(over.argmax(), over.shape)}"
                               f" by {np.abs(got - want['out']).max():.3g}, tolerance {tol.flat[over.argmax()]:.3g}")
    if weights:
        rows = queries * heads // kv_heads
        wtol = want["weights"] * (2 * delta.max() + (rows + 8) * 2.0 ** -23) + 2.0 ** -23 * (w0 + want["weights"])
        diff = np.abs(w.double().cpu().numpy() - (w0.astype(np.float64) + want["weights"]))
        assert (diff <= wtol).all(), f"weights: {(diff > wtol).sum()} of {diff.size} off, by {diff.max():.3g}"
    _same_cache(cache, c, "attention leaves the cache alone")
    return out


HEADS = [(2, 1, 64), (16, 8, 256), (4, 4, 128), (16, 2, 64), (10, 2, 128), (8, 1, 256), (3, 1, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("queries,lengths", [(1, [1, 64, 65]), (1, [0, 700, 513]), (2, [2, 1, 130]), (5, [300, 5, 64])])
def test_attention_few_queries(queries, lengths, heads, kv_heads, dim, weights, dtype):
    rng = np.random.default_rng(dim + heads + sum(lengths))
    c = ref.make_cache(rng, 3, kv_heads, dim, lengths, max(1, -(-max(lengths) // PAGE)))
    _check_attention(c, 3, queries, heads, dtype, [min(queries, n) for n in lengths], weights, seed=1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("queries,lengths,weights", [(33, [33, 200], False), (70, [70, 65], True), (129, [129, 400], False),
                                                     (40, [1000, 41], True)])
def test_attention_prompts(queries, lengths, weights, heads, kv_heads, dim, dtype):
    rng = np.random.default_rng(dim + heads + sum(lengths))
    c = ref.make_cache(rng, 2, kv_heads, dim, lengths, -(-max(lengths) // PAGE))
    _check_attention(c, 2, queries, heads, dtype, [min(queries, n) for n in lengths], weights, seed=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 3, 40])
def test_attention_rows_that_see_nothing(queries, dtype):
    """Empty sequences, no queries, more queries than tokens, pages that are not there (all of a sequence's, its first, its
    last): such rows are zeros, the others as if the tokens were not."""
    rng = np.random.default_rng(9)
    lengths = [0, 100, 2, 128, 192, 190, 500]
    c = ref.make_cache(rng, 7, 2, 64, lengths, 8, absent=[(3, 0), (3, 1), (4, 0), (5, 2), (6, 3), (6, 6)])
    lens = [queries, 0, queries, queries, queries, queries, queries]
    out = _check_attention(c, 7, queries, 4, dtype, lens, True, seed=3)
    assert (out[0] == 0).all() and (out[1] == 0).all() and (out[3] == 0).all()


@pytest.mark.parametrize("queries", [1, 40])
def test_pages_given_ahead_do_not_matter(queries):
    """Table entries behind a sequence's end may name pages that hold nothing yet (NaN scales)."""
    rng = np.random.default_rng(14)
    c = ref.make_cache(rng, 4, 2, 128, [0, 1, 64, 300], 9, ahead=True)
    _check_attention(c, 4, queries, 4, torch.bfloat16, [0, 1, min(queries, 64), queries], True, seed=7)
    k, v = qar.qar_kv8_read(ref.to_cache(c), _ints(0, 0, 0, 0), 400, out_dtype=torch.float32)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_lengths_out_of_range(dtype):
    """Lengths beyond the table and below zero are clipped, q_lens likewise."""
    rng = np.random.default_rng(10)
    c = ref.make_cache(rng, 3, 1, 128, [128, 128, 128], 2)
    c["lengths"][:] = [2 ** 31 - 1, -5, 129]
    for queries in (2, 50):
        _check_attention(c, 3, queries, 2, dtype, [2 ** 31 - 1, -3, 1], True, seed=4)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 40])
def test_attention_scales_far_apart(queries, dtype):
    """Page scales that differ by 2^60 and pages of zeros; queries from subnormal to huge; peaked and flat softmaxes."""
    rng = np.random.default_rng(11)
    c = ref.make_cache(rng, 2, 2, 64, [640, 333], 10)
    ids = [i for i in c["page_table"].ravel() if i >= 0]
    for n, i in enumerate(ids):
        c["v_scales"][i] *= np.float32(2.0 ** (n * 37 % 60 - 30))
        if n % 5 == 4:
            c["k_scales"][i] = 0
            c["v_scales"][i, 0] = 0
    for spread, scale in ((1e-30, 1e30), (1e-41, 1.0), (1e4, 1e-4), (30.0, None), (0.0, None)):
        _check_attention(c, 2, queries, 4, dtype, None, True, scale=scale, seed=5, spread=spread)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries,heads,n", [(1, 4, 70), (2, 4, 6000), (40, 4, 200), (70, 2, 3000)])
def test_attention_keeps_a_nan_to_its_row(queries, heads, n, dtype):
    rng = np.random.default_rng(15)
    c = ref.make_cache(rng, 1, 2, 128, [n], -(-n // PAGE))
    q, values = ref.data(rng, (1, queries, heads, 128), dtype)
    want = ref.attend(c, values, [queries], 128 ** -0.5)
    tol, _ = _attention_tolerance(want, q, dtype, 128, n)
    q[0, -1, 1, 77] = float("nan")
    got = qar.qar_kv8_attention(ref.to_cache(c), q).double().cpu().numpy()
    assert np.isnan(got[0, -1, 1]).all()
    got[0, -1, 1] = want["out"][0, -1, 1]
    assert (np.abs(got - want["out"]) <= tol).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("batch,kv_heads,heads,dim,queries,n", [(1, 1, 1, 64, 1, 20000), (1, 2, 16, 64, 3, 9000),
                                                               (1, 1, 8, 128, 60, 5000), (40, 8, 8, 64, 1, 300)])
def test_attention_split_over_long_caches(batch, kv_heads, heads, dim, queries, n, dtype):
    rng = np.random.default_rng(n)
    lengths = [n] + [int(v) for v in rng.integers(1, n, batch - 1)]
    c = ref.make_cache(rng, batch, kv_heads, dim, lengths, -(-n // PAGE))
    _check_attention(c, batch, queries, heads, dtype, [min(queries, v) for v in lengths], True, seed=6)


def test_attention_repeats_bit_for_bit_on_any_workspace():
    rng = np.random.default_rng(12)
    c = ref.make_cache(rng, 2, 2, 128, [1500, 900], 24)
    cache = ref.to_cache(c)
    for queries in (1, 50):
        q, _ = ref.data(rng, (2, queries, 8, 128), torch.bfloat16)
        need = qar.lib().qar_kv8_attention_workspace_bytes(2, queries, 8, 2, 128, 24, 0, 1)
        assert need > 0
        outs, sums = [], []
        for fill in (0, 255, 127):
            w = torch.zeros((2, 2, 24 * PAGE), device=DEV)
            outs.append(qar.qar_kv8_attention(cache, q, weights=w,
                                              workspace=torch.full((need,), fill, dtype=torch.uint8, device=DEV)))
            sums.append(w)
        assert all(torch.equal(outs[0], o) for o in outs) and all(torch.equal(sums[0], w) for w in sums)


# ---------------------------------------------------------------------------
# eviction


@pytest.mark.parametrize("heads,dim,lengths,keep,recent", [
    (1, 64, [1], 1, 0), (2, 128, [100, 64, 0], 64, 10), (1, 256, [300, 299], 130, 130), (2, 64, [500, 20], 499, 0),
    (3, 64, [1000, 65, 700], 65, 200), (1, 128, [3000, 2999, 1], 777, 64), (1, 64, [129], 1, 5), (1, 64, [5000], 2048, 1)])
@pytest.mark.parametrize("kind", ["normal", "ties", "special"])
def test_evict(heads, dim, lengths, keep, recent, kind):
    rng = np.random.default_rng(keep + dim)
    batch, width = len(lengths), max(1, -(-max(lengths) // PAGE))
    c = ref.make_cache(rng, batch, heads, dim, lengths, width, absent=[(0, 1)] if width > 3 else ())
    out = -(-keep // PAGE) + 1
    d = ref.make_cache(rng, batch, heads, dim, [keep] * batch, out)
    d["k_scales"][:], d["v_scales"][:] = 5, 5
    w = rng.standard_normal((batch, heads, width * PAGE)).astype(np.float32)
    if kind == "ties":
        w = np.round(w)
    elif kind == "special":
        w[rng.random(w.shape) < 0.2] = 0.0
        w[rng.random(w.shape) < 0.2] = -0.0
        w[rng.random(w.shape) < 0.05] = np.inf
        w[rng.random(w.shape) < 0.05] = -np.inf
        w[rng.random(w.shape) < 0.05] = 1e-42
        w[rng.random(w.shape) < 0.02] = np.nan
    cache, into = ref.to_cache(c), ref.to_cache(d)
    kept, moved = qar.qar_kv8_evict(cache, into, _dev(w), recent, keep)
    want, wmoved = ref.evict(c, d, w, recent, keep)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(moved.cpu().numpy(), wmoved, equal_nan=True)
    _same_cache(into, d, "into", [min(n, keep) for n in lengths])
    _same_cache(cache, c, "evict leaves the source alone")


@pytest.mark.parametrize("lengths,keep,recent", [([2048, 2047], 2000, 3), ([2049, 600], 1000, 100), ([8192, 8000], 100, 0),
                                                 ([8193, 700], 4096, 1000), ([24577, 24576], 5000, 64), ([40000], 39999, 0)])
def test_evict_long_caches(lengths, keep, recent):
    """Lengths around what a workgroup's threads hold of a sequence."""
    rng = np.random.default_rng(lengths[0])
    c = ref.make_cache(rng, len(lengths), 1, 64, lengths, -(-max(lengths) // PAGE))
    d = ref.make_cache(rng, len(lengths), 1, 64, [keep] * len(lengths), -(-keep // PAGE))
    w = np.round(rng.standard_normal((len(lengths), 1, c["page_table"].shape[1] * PAGE)) * 300).astype(np.float32)
    into = ref.to_cache(d)
    kept, moved = qar.qar_kv8_evict(ref.to_cache(c), into, _dev(w), recent, keep)
    want, wmoved = ref.evict(c, d, w, recent, keep)
    assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(moved.cpu().numpy(), wmoved)
    _same_cache(into, d, "into", [min(n, keep) for n in lengths])


def test_evict_leaves_out_pages_that_are_not_there():
    rng = np.random.default_rng(20)
    c = ref.make_cache(rng, 2, 2, 64, [400, 390], 7, absent=[(0, 2), (1, 0)])
    d = ref.make_cache(rng, 2, 2, 64, [256, 256], 4, absent=[(0, 1), (1, 3)])
    w = rng.uniform(0, 1, (2, 2, 7 * PAGE)).astype(np.float32)
    into = ref.to_cache(d)
    qar.qar_kv8_evict(ref.to_cache(c), into, _dev(w), 32, 200)
    ref.evict(c, d, w, 32, 200)
    _same_cache(into, d, "into", [200, 200])


def test_evict_within_one_pool():
    """cache and into may share a pool; their pages are disjoint."""
    rng = np.random.default_rng(21)
    c = ref.make_cache(rng, 1, 2, 64, [256], 8)
    free = np.array([i for i in range(c["k"].shape[0]) if i not in c["page_table"]], np.int32)
    d = dict(c, page_table=free[None, :2].copy(), lengths=np.zeros(1, np.int32))
    cache = ref.to_cache(c)
    into = qar.KvCache(cache.k, cache.k_scales, cache.v, cache.v_scales, _dev(d["page_table"]), _ints(0))
    w = rng.uniform(0, 1, (1, 2, 8 * PAGE)).astype(np.float32)
    qar.qar_kv8_evict(cache, into, _dev(w), 10, 100)
    ref.evict(c, d, w, 10, 100)
    _same_cache(into, d, "into", [100])


# ---------------------------------------------------------------------------
# streams, graphs, empty calls


def test_a_step_on_a_stream_and_in_a_graph():
    """append, attention with weights and evict captured together; every replay equals the eager calls on the same data."""
    rng = np.random.default_rng(30)
    c = ref.make_cache(rng, 2, 2, 64, [200, 131], 4)
    c["k_scales"][np.isnan(c["k_scales"])] = 1
    d = ref.make_cache(rng, 2, 2, 64, [128, 128], 2)
    k, _ = ref.data(rng, (2, 1, 2, 64), torch.bfloat16)
    q, _ = ref.data(rng, (2, 1, 4, 64), torch.bfloat16)
    need = qar.lib().qar_kv8_attention_workspace_bytes(2, 1, 4, 2, 64, 4, 0, 1)
    ws = torch.empty(max(256, need), dtype=torch.uint8, device=DEV)
    starts = _ints(199, 130)

    def fresh():
        return ref.to_cache(c), ref.to_cache(d), torch.zeros((2, 2, 256), device=DEV), torch.empty_like(q), \
            torch.empty((2, 2, 100), dtype=torch.int32, device=DEV), torch.empty((2, 2, 100), device=DEV)

    def step(s, stream=None):
        qar.qar_kv8_append(s[0], starts, k, k, stream=stream)
        qar.qar_kv8_attention(s[0], q, weights=s[2], out=s[3], workspace=ws, stream=stream)
        qar.qar_kv8_evict(s[0], s[1], s[2], 16, 100, kept=s[4], moved=s[5], stream=stream)

    def equal(a, b):
        assert all(torch.equal(x, y) for x, y in zip(a[2:], b[2:]))
        for x, y in zip(a[:2], b[:2]):
            for name in ("k", "v", "lengths"):
                assert torch.equal(getattr(x, name), getattr(y, name)), name
            for name in ("k_scales", "v_scales"):
                assert torch.equal(torch.nan_to_num(getattr(x, name)), torch.nan_to_num(getattr(y, name))), name

    eager, sided, graphed = fresh(), fresh(), fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(sided, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for i in range(4):
        if i:
            k.copy_(ref.data(rng, k.shape, torch.bfloat16)[0])
            q.copy_(ref.data(rng, q.shape, torch.bfloat16)[0])
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        equal(eager, graphed)
        if i == 0:
            equal(eager, sided)


def test_memory_of_a_call_on_another_stream_is_not_reused_under_it():
    """Workspace and outputs that a call on a side stream allocates belong to that stream: work on the main stream that asks
    for memory of the same sizes meanwhile does not get it."""
    rng = np.random.default_rng(32)
    cache = ref.to_cache(ref.make_cache(rng, 1, 1, 64, [30000], 469))
    q, _ = ref.data(rng, (1, 2, 4, 64), torch.bfloat16)
    want = qar.qar_kv8_attention(cache, q)
    need = qar.lib().qar_kv8_attention_workspace_bytes(1, 2, 4, 1, 64, 469, 0, 0)
    assert need > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        for _ in range(20):
            got = qar.qar_kv8_attention(cache, q, stream=handle)
            for _ in range(4):
                torch.empty(need, dtype=torch.uint8, device=DEV).fill_(255)
            side.synchronize()
            assert torch.equal(got, want)


def test_empty_calls():
    rng = np.random.default_rng(31)
    cache = ref.to_cache(ref.make_cache(rng, 2, 1, 64, [10, 0], 1))
    x = torch.empty((2, 0, 1, 64), device=DEV)
    qar.qar_kv8_append(cache, _ints(0, 0), x, x)
    assert qar.qar_kv8_read(cache, _ints(0, 0), 0)[0].shape == (2, 0, 1, 64)
    assert qar.qar_kv8_attention(cache, x).shape == (2, 0, 1, 64)


def test_stale_runtime_error_does_not_fail_a_good_call():
    """A launch reports its own status: an error that an unrelated HIP call left on the thread (an invalid hipSetDevice) must
    not turn a valid call into QAR_ERR_HIP."""
    import ctypes
    maps = open("/proc/self/maps").read().split()
    hip = ctypes.CDLL(next(p for p in maps if "libamdhip64.so" in p))
    hip.hipSetDevice.argtypes = [ctypes.c_int]
    rng = np.random.default_rng(33)
    c = ref.make_cache(rng, 2, 2, 64, [200, 131], 4)
    cache, into = ref.to_cache(c), ref.to_cache(ref.make_cache(rng, 2, 2, 64, [128, 128], 2))
    k, _ = ref.data(rng, (2, 1, 2, 64), torch.bfloat16)
    outs = qar.qar_kv8_read(cache, _ints(0, 0), 100)
    starts, kept = _ints(199, 130), torch.empty((2, 2, 100), dtype=torch.int32, device=DEV)
    moved, summed = torch.empty((2, 2, 100), device=DEV), torch.zeros((2, 2, 256), device=DEV)
    x, _ = ref.data(rng, (90, 200), torch.bfloat16)
    w, s = qar.qar_mx4_quantize(x)
    calls = [lambda: qar.qar_kv8_append(cache, starts, k, k), lambda: qar.qar_kv8_read(cache, starts, 100, out=outs),
             lambda: qar.qar_kv8_evict(cache, into, summed, 16, 100, kept=kept, moved=moved),
             lambda: qar.qar_mx4_quantize(x, codes=w, scales=s)]
    for queries in (1, 50):
        q, _ = ref.data(rng, (2, queries, 4, 64), torch.bfloat16)
        need = qar.lib().qar_kv8_attention_workspace_bytes(2, queries, 4, 2, 64, 4, 0, 1)
        ws, out = torch.empty(max(256, need), dtype=torch.uint8, device=DEV), torch.empty_like(q)
        calls.append(lambda q=q, ws=ws, out=out: qar.qar_kv8_attention(cache, q, weights=summed, out=out, workspace=ws))
    for rows in (4, 20, 90):
        ws = torch.empty(max(256, qar.lib().qar_mx4_linear_workspace_bytes(rows, 200, 90)), dtype=torch.uint8, device=DEV)
        y = torch.empty((rows, 90), dtype=torch.bfloat16, device=DEV)
        calls.append(lambda a=x[:rows], y=y, ws=ws: qar.qar_mx4_linear(a, w, s, out=y, workspace=ws))
    y = torch.empty_like(x)
    calls.append(lambda: qar.qar_mx4_dequantize(w, s, 200, out=y))
    torch.cuda.synchronize()
    for call in calls:
        assert hip.hipSetDevice(1 << 20) != 0                # hipErrorInvalidDevice, left on the thread
        try:
            call()
        finally:
            hip.hipGetLastError()                            # clear what the test left behind
    torch.cuda.synchronize()
