"""Attention behind shared prefixes on the GPU, against tests/serve_reference.py's attention of each sequence for itself."""
import numpy as np
import pytest
import serve_reference as ref
import torch
from test_gpu_kv8 import HEADS, _attention_tolerance, _ints, _same_cache

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64
DTYPES = [torch.bfloat16, torch.float32]


def _shared_cache(rng, kv_heads, dim, starts, prefix, lengths, width, absent=(), spare=3):
    """A cache whose groups name the same pages for the whole pages of their prefix."""
    c = ref.make_cache(rng, len(lengths), kv_heads, dim, lengths, width, spare=spare, ahead=True)
    for g in range(len(starts) - 1):
        whole = min(max(prefix[g], 0) // PAGE, width)
        for b in range(starts[g], starts[g + 1]):
            c["page_table"][b, :whole] = c["page_table"][starts[g], :whole]
    # pages that no sequence has tokens in hold NaN scales, the others none
    used = np.zeros(c["k"].shape[0], bool)
    for b, n in enumerate(lengths):
        used[c["page_table"][b, :-(-min(max(n, 0), width * PAGE) // PAGE)]] = True
    for name in ("k_scales", "v_scales"):
        c[name][used] = (rng.uniform(0.5, 2, (used.sum(), kv_heads)) / 127).astype(np.float32)
        c[name][~used] = np.nan
    for b, p in absent:
        c["page_table"][b, p] = [c["k"].shape[0], -7, 2 ** 31 - 1, -2 ** 31][(b + p) % 4]
    return c


def _check(c, starts, prefix, queries, heads, dtype, q_lens=None, scale=None, seed=0, spread=1.5, q=None, workspace=None):
    rng = np.random.default_rng(seed)
    batch, dim = len(c["lengths"]), c["k"].shape[3]
    if q is None:
        q = torch.from_numpy(rng.standard_normal((batch, queries, heads, dim)).astype(np.float32)) * spread
    q = q.to(dtype)
    lens = [queries] * batch if q_lens is None else q_lens
    want = ref.attend(c, q.float().numpy(), lens, dim ** -0.5 if scale is None else scale)
    cache = ref.to_cache(c)
    out = qar.qar_kv8_attention_shared(cache, q.to(DEV), _ints(*starts), _ints(*prefix),
                                       q_lens=None if q_lens is None else _ints(*q_lens), scale=scale, workspace=workspace)
    # the arithmetic is qar_kv8_attention's; joining two more partial sums adds less than its allowance for n additions
    tol, _ = _attention_tolerance(want, q, dtype, dim, int(max(0, c["lengths"].max())) + PAGE)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - want["out"]) - tol
    assert (over <= 0).all(), (f"{(over > 0).sum()} of {over.size} off, worst at {np.unravel_index(over.argmax(), over.shape)}"
                               f" by {np.abs(got - want['out']).max():.3g}, tolerance {tol.flat[over.argmax()]:.3g}")
    _same_cache(cache, c, "attention leaves the cache alone")
    return out


GROUPS = [([0, 3], [130], [131, 200, 320]),                            # one group; a prefix that ends inside a page
          ([0, 1, 2, 5], [64, 200, 256], [65, 201, 257, 300, 500]),    # alone, alone, three
          ([0, 9], [640], [641 + 13 * i for i in range(9)]),
          ([0, 4, 12], [63, 128], [64 + i for i in range(4)] + [129 + 30 * i for i in range(8)])]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("queries", [1, 2])
@pytest.mark.parametrize("starts,prefix,lengths", GROUPS)
def test_single_tokens(starts, prefix, lengths, queries, heads, kv_heads, dim, dtype):
    rng = np.random.default_rng(dim + heads + sum(lengths))
    c = _shared_cache(rng, kv_heads, dim, starts, prefix, [n + queries for n in lengths], -(-(max(lengths) + queries) // PAGE))
    _check(c, starts, prefix, queries, heads, dtype, seed=1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("queries,starts,prefix,lengths", [
    (40, [0, 3], [130], [190, 180, 301]), (70, [0, 2, 3], [64, 128], [140, 200, 198]), (129, [0, 2], [300], [429, 500])])
def test_prompts_that_go_on(queries, starts, prefix, lengths, heads, kv_heads, dim, dtype):
    """Many queries of each sequence, causal among its own tokens."""
    rng = np.random.default_rng(dim + heads + sum(lengths))
    c = _shared_cache(rng, kv_heads, dim, starts, prefix, lengths, -(-max(lengths) // PAGE))
    _check(c, starts, prefix, queries, heads, dtype, seed=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 3, 50])
@pytest.mark.parametrize("dim", [64, 128])
def test_lengths_and_groups_of_every_kind(queries, dim, dtype):
    """Empty sequences, no queries, more queries than tokens, sequences that end inside or before their prefix, sequences
    outside every group, an empty group, prefixes below 0, of 0, up to a length, behind the table."""
    rng = np.random.default_rng(9)
    starts, prefix = [1, 4, 4, 6, 9, 11, 12], [200, 128, -5, 10_000, 0, 64]
    lengths = [70, 300, 150, 0, 90, 1, 300, 512, 640, 100, 30, 64, 333]
    lens = [queries, queries, 0, queries, queries, queries, queries, queries, max(1, queries - 1), queries, queries, queries, queries]
    c = _shared_cache(rng, 2, dim, starts, prefix, lengths, 10)
    out = _check(c, starts, prefix, queries, 4, dtype, lens, seed=3)
    assert (out[2] == 0).all() and (out[3] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 40])
def test_absent_pages(queries, dtype):
    """Pages that are not there: in a prefix (all, the first, some), among own tokens."""
    rng = np.random.default_rng(10)
    starts, prefix = [0, 2, 4, 6], [192, 128, 320]
    lengths = [300, 260, 190, 200, 321, 500]
    absent = [(b, p) for b in (0, 1) for p in (0, 2)] + [(b, p) for b in (2, 3) for p in (0, 1)] + [(4, 3), (5, 3), (5, 6), (2, 2)]
    c = _shared_cache(rng, 2, 64, starts, prefix, lengths, 8, absent=absent)
    _check(c, starts, prefix, queries, 4, dtype, seed=4)


@pytest.mark.parametrize("members,heads,kv_heads,dim,prefix", [
    (64, 32, 8, 128, 1000), (40, 64, 8, 64, 2100), (33, 8, 1, 256, 700), (9, 14, 2, 128, 5000), (128, 4, 4, 64, 300),
    (16, 16, 8, 256, 1500)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_large_groups(members, heads, kv_heads, dim, prefix, dtype):
    """Several tiles of rows, many slots of pages, tiles that end between and inside sequences."""
    rng = np.random.default_rng(members)
    lengths = [prefix + 1 + int(n) for n in rng.integers(0, 200, members)]
    c = _shared_cache(rng, kv_heads, dim, [0, members], [prefix], lengths, -(-max(lengths) // PAGE) + 1)
    _check(c, [0, members], [prefix], 1, heads, dtype, seed=5)


def test_many_groups():
    """More groups than a wave looks at at once, some without sequences."""
    rng = np.random.default_rng(11)
    sizes = [int(n) for n in rng.integers(0, 4, 150)]
    starts = np.concatenate(([2], 2 + np.cumsum(sizes))).tolist()
    batch = starts[-1] + 3
    prefix = [int(n) for n in rng.integers(0, 300, len(sizes))]
    of = {b: g for g in range(len(sizes)) for b in range(starts[g], starts[g + 1])}
    lengths = [(prefix[of[b]] if b in of else 0) + int(rng.integers(1, 100)) for b in range(batch)]
    c = _shared_cache(rng, 1, 64, starts, prefix, lengths, 7)
    for dtype in DTYPES:
        _check(c, starts, prefix, 1, 3, dtype, seed=6)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scales_far_apart_and_steep_scores(dtype):
    rng = np.random.default_rng(12)
    starts, prefix, lengths = [0, 40], [700], [701 + i for i in range(40)]
    c = _shared_cache(rng, 2, 64, starts, prefix, lengths, 13)
    c["v_scales"] *= np.exp2(rng.integers(-30, 31, c["v_scales"].shape)).astype(np.float32)
    _check(c, starts, prefix, 1, 4, dtype, seed=7)
    c["v_scales"][:] = np.where(np.isnan(c["v_scales"]), c["v_scales"], np.float32(0))
    _check(c, starts, prefix, 1, 4, dtype, seed=7)
    c = _shared_cache(rng, 2, 64, starts, prefix, lengths, 13)
    c["k_scales"] *= np.exp2(rng.integers(-20, 4, c["k_scales"].shape)).astype(np.float32)
    _check(c, starts, prefix, 1, 4, dtype, scale=-0.3, seed=8, spread=4.0)
    _check(c, starts, prefix, 1, 4, dtype, scale=0.0, seed=8)


def test_a_nan_stays_in_its_row():
    rng = np.random.default_rng(13)
    starts, prefix, lengths = [0, 20], [300], [301 + i for i in range(20)]
    c = _shared_cache(rng, 2, 64, starts, prefix, lengths, 6)
    cache = ref.to_cache(c)
    q = torch.from_numpy(rng.standard_normal((20, 2, 8, 64)).astype(np.float32)).to(DEV)
    for dtype in DTYPES:
        clean = qar.qar_kv8_attention_shared(cache, q.to(dtype), _ints(0, 20), _ints(300))
        bad = q.to(dtype).clone()
        bad[7, 1, 3, 5] = float("nan")
        got = qar.qar_kv8_attention_shared(cache, bad, _ints(0, 20), _ints(300))
        rows = torch.isnan(got).all(3)
        assert rows[7, 1, 3] and rows.sum() == 1
        assert torch.equal(got[~rows], clean[~rows])


@pytest.mark.parametrize("heads,kv_heads,dim,members", [(16, 2, 128, 8), (8, 2, 256, 8), (8, 2, 256, 20),
                                                           (2, 2, 128, 80)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_many_rows_over_absent_pages_and_scales_far_apart(heads, kv_heads, dim, members, dtype):
    """What the bodies for many rows do a page ahead: the next page may be absent, the last one or in another unit."""
    rng = np.random.default_rng(dim + members)
    for pages in (1, 2, 3, 5, 12):
        prefix = 64 * pages + 20
        lengths = [prefix + 1 + i for i in range(members)]
        absent = [(b, p) for b in range(members) for p in range(pages) if pages > 3 and p % 5 in (0, 3)]
        c = _shared_cache(rng, kv_heads, dim, [0, members], [prefix], lengths, pages + 3, absent=absent)
        c["v_scales"] *= np.exp2(rng.integers(-30, 31, c["v_scales"].shape)).astype(np.float32)
        c["k_scales"] *= np.exp2(rng.integers(-6, 2, c["k_scales"].shape)).astype(np.float32)
        _check(c, [0, members], [prefix], 1, heads, dtype, seed=pages)
        _check(c, [0, members], [prefix], 20, heads, dtype, seed=pages, scale=-0.05)


@pytest.mark.parametrize("dtype", DTYPES)
def test_more_pages_than_are_looked_up_at_once(dtype):
    """256 tiles of own rows: one slot of up to 70 pages each.  One head of two sequences is compared."""
    rng = np.random.default_rng(16)
    c = _shared_cache(rng, 8, 128, [0, 4], [128], [64 * 70 - 5, 64 * 69, 64 * 66 + 1, 4000], 70)
    q = torch.from_numpy(rng.standard_normal((4, 1024, 8, 128)).astype(np.float32)).to(dtype)
    out = qar.qar_kv8_attention_shared(ref.to_cache(c), q.to(DEV), _ints(0, 4), _ints(128)).double().cpu().numpy()
    part = {**c, **{n: np.ascontiguousarray(c[n][:, 5:6]) for n in ("k", "v", "k_scales", "v_scales")}}
    for b in (0, 1):
        one = {**part, "page_table": c["page_table"][b:b + 1], "lengths": c["lengths"][b:b + 1]}
        mine = q[b:b + 1, :, 5:6]
        want = ref.attend(one, mine.float().numpy(), [1024], 128 ** -0.5)
        tol, _ = _attention_tolerance(want, mine, dtype, 128, int(c["lengths"][b]) + PAGE)
        assert (np.abs(out[b:b + 1, :, 5:6] - want["out"]) <= tol).all()


def test_a_nan_stays_in_its_row_of_many():
    rng = np.random.default_rng(17)
    c = _shared_cache(rng, 2, 128, [0, 20], [900], [901 + i for i in range(20)], 16)
    cache = ref.to_cache(c)
    q = torch.from_numpy(rng.standard_normal((20, 2, 8, 128)).astype(np.float32)).to(DEV)
    for dtype in DTYPES:
        clean = qar.qar_kv8_attention_shared(cache, q.to(dtype), _ints(0, 20), _ints(900))
        bad = q.to(dtype).clone()
        bad[7, 1, 3, 5] = float("nan")
        got = qar.qar_kv8_attention_shared(cache, bad, _ints(0, 20), _ints(900))
        rows = torch.isnan(got).all(3)
        assert rows[7, 1, 3] and rows.sum() == 1
        assert torch.equal(got[~rows], clean[~rows])


def test_equal_calls_and_workspaces():
    """Equal bits whatever the workspace held; nothing behind the output or the workspace's stated end is written."""
    rng = np.random.default_rng(14)
    starts, prefix, lengths = [0, 6, 9], [500, 200], [501 + 40 * i for i in range(6)] + [210, 260, 500]
    c = _shared_cache(rng, 2, 128, starts, prefix, lengths, 12)
    cache = ref.to_cache(c)
    for queries, heads in ((1, 4), (1, 40), (60, 4)):
        q = torch.from_numpy(rng.standard_normal((9, queries, heads, 128)).astype(np.float32)).to(DEV)
        need = qar.lib().qar_kv8_attention_shared_workspace_bytes(9, queries, heads, 2, 128, 12, 2)
        got = []
        for fill in (0, 255, 17):
            ws = torch.full((need + 1024,), fill, dtype=torch.uint8, device=DEV)
            flat = torch.full((q.numel() + 64,), 7.0, device=DEV)
            got.append(qar.qar_kv8_attention_shared(cache, q, _ints(*starts), _ints(*prefix), workspace=ws[:need],
                                                    out=flat[:q.numel()].view(q.shape)))
            assert (ws[need:] == fill).all() and (flat[q.numel():] == 7).all()
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_streams_and_graphs():
    """Captured, with lengths, groups and prefixes that change between the replays."""
    rng = np.random.default_rng(15)
    starts, prefix, lengths = [0, 6, 9], [500, 200], [520 + 20 * i for i in range(6)] + [210, 260, 500]
    c = _shared_cache(rng, 2, 64, starts, prefix, lengths, 12)
    cache = ref.to_cache(c)
    st, pf = _ints(*starts), _ints(*prefix)
    for queries in (1, 40):
        q = torch.from_numpy(rng.standard_normal((9, queries, 8, 64)).astype(np.float32)).to(DEV).bfloat16()
        want = qar.qar_kv8_attention_shared(cache, q, st, pf)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = qar.qar_kv8_attention_shared(cache, q, st, pf, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = qar.qar_kv8_attention_shared(cache, q, st, pf)
        for step in range(4):
            q.copy_(torch.randn_like(q))
            cache.lengths -= 3
            pf.copy_(_ints(500 - 64 * step, 128))
            st.copy_(_ints(0, 6 - step, 6 - step))
            if step == 3:
                st.copy_(_ints(*starts))
            want = qar.qar_kv8_attention_shared(cache, q, st, pf)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want), (queries, step)
        cache.lengths += 12
        pf.copy_(_ints(*prefix))


def test_it_agrees_with_attention_of_each_for_itself():
    """A long prefix: the two kernels' results differ by less than both their roundings."""
    rng = np.random.default_rng(16)
    lengths = [20_001 + 50 * i for i in range(12)]
    c = _shared_cache(rng, 2, 128, [0, 12], [20_000], lengths, 330)
    cache = ref.to_cache(c)
    q = torch.from_numpy(rng.standard_normal((12, 1, 8, 128)).astype(np.float32)).to(DEV)
    a, b = qar.qar_kv8_attention(cache, q), qar.qar_kv8_attention_shared(cache, q, _ints(0, 12), _ints(20_000))
    # scores of up to some 6, each off by 136 units of 2^-23 of their magnitudes at most in either
    assert ((a - b).abs() <= 2 * 136 * 2.0 ** -23 * 40 * a.abs().max()).all()
