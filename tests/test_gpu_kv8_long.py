"""Attention where a wave runs over many pages and prompts over many tiles, against a 64-bit softmax on the GPU.

The cuts that test_gpu_kv8.py does not reach: more than 64 pages to a workgroup of a prompt and more than 256 to one of few
rows (page numbers are looked up 64 at a time by every wave), alone and as one of several cuts; tiles of prompts enough for
the sequences to be turned over the CUs.  Sequences share the pool's pages, which attention only reads.
"""
import numpy as np
import pytest
import serve_reference as ref
import torch

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64
BF16, F32 = torch.bfloat16, torch.float32


def _cache(rng, lengths, kv_heads, dim, absent=(), spread=0, pages=300):
    """A pool whose pages the sequences share, in any order; behind a sequence's end the table names nothing.  `absent`: page
    numbers that are not there in any sequence.  `spread`: the pages' value scales differ by up to 2^spread."""
    g = torch.Generator(device=DEV).manual_seed(int(rng.integers(1 << 30)))
    shape = (pages, kv_heads)
    k = torch.randint(-127, 128, (*shape, PAGE, dim), generator=g, device=DEV, dtype=torch.int8)
    v = torch.randint(-127, 128, (*shape, dim, PAGE), generator=g, device=DEV, dtype=torch.int8)
    ks, vs = ((torch.rand(shape, generator=g, device=DEV) * 1.5 + 0.5) / 127 for _ in range(2))
    if spread:
        vs *= torch.exp2(torch.randint(-(spread // 2), spread // 2 + 1, shape, generator=g, device=DEV).float())
    width = -(-max(lengths) // PAGE)
    table = rng.integers(0, pages, (len(lengths), width)).astype(np.int32)
    for b, n in enumerate(lengths):
        table[b, -(-n // PAGE):] = -1
    for p in absent:
        if p < width:
            table[:, p] = pages + p
    return qar.KvCache(k, ks, v, vs, torch.from_numpy(table).to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV))


def _check(cache, q, q_lens, weights):
    """Outputs and weights within what the arithmetic can do to a row.  A score is a sum of `dim` exact products in binary32
    (binary32 queries off by 2^-23 of an element) and a few roundings, so off by (dim + 8) 2^-23 of its magnitudes' sum, and
    its exponential by that and 2^-20; the softmax's sum doubles this.  A numerator enters the product rounded to 2^-12 (bf16)
    or 2^-22 (binary32); sums over n keys add n 2^-24.  Numerators enter times 2^14 and their page's scale ratio: below 2^-28
    of the row's largest they are binary16 subnormals, off by 2^-39 of the largest value each.  A weight is a sum over rows of
    such exponentials, each divided by a sum over n keys, added to what was there."""
    batch, queries, heads, dim = q.shape
    kv_heads = cache.k.shape[1]
    group = heads // kv_heads
    before = [t.clone() for t in (cache.k, cache.k_scales, cache.v, cache.v_scales, cache.page_table, cache.lengths)]
    w0 = None
    if weights:
        w0 = torch.rand((batch, kv_heads, cache.page_table.shape[1] * PAGE), device=DEV)
    w = None if w0 is None else w0.clone()
    lens = torch.tensor(q_lens, dtype=torch.int32, device=DEV)
    out = qar.qar_kv8_attention(cache, q, q_lens=lens, weights=w)
    assert torch.isfinite(out).all()
    scale, rounding = dim ** -0.5, 2.0 ** -12 if q.dtype == BF16 else 2.0 ** -22
    for b in range(batch):
        n, m = int(cache.lengths[b]), q_lens[b]
        assert (out[b, m:] == 0).all()
        ids = cache.page_table[b, :-(-n // PAGE)].long()
        there = ((ids >= 0) & (ids < cache.k.shape[0])).repeat_interleave(PAGE)[:n]
        ids = ids.clamp(0, cache.k.shape[0] - 1)
        sees = torch.arange(n, device=DEV)[None] < (n - m + 1 + torch.arange(m, device=DEV))[:, None]
        sees = (sees & there).repeat_interleave(group, 0)
        for h in range(kv_heads):
            k = (cache.k[ids, h].double() * cache.k_scales[ids, h].double()[:, None, None]).reshape(-1, dim)[:n]
            v = (cache.v[ids, h].double() * cache.v_scales[ids, h].double()[:, None, None]).transpose(1, 2).reshape(-1, dim)[:n]
            rows = q[b, :m, h * group:(h + 1) * group].double().reshape(m * group, dim)
            got = out[b, :m, h * group:(h + 1) * group].double().reshape(m * group, dim)
            if m == 0 or n == 0:
                continue
            s = (rows @ k.T * scale).masked_fill(~sees, -torch.inf)
            top = s.amax(1, keepdim=True)
            p = torch.exp(s - torch.where(top > -torch.inf, top, 0.0))
            total = p.sum(1, keepdim=True)
            p = p / torch.where(total > 0, total, 1.0)
            delta = (dim + 8) * 2.0 ** -23 * scale * (rows.abs() @ k.abs().T).masked_fill(~sees, 0).amax(1) + 2.0 ** -20
            largest = v.abs().amax()
            want = p @ v
            tol = ((2 * delta + rounding + (n + 8) * 2.0 ** -24)[:, None] * (p @ v.abs()) + ref.half_step(q.dtype) * want.abs()
                   + n * 2.0 ** -39 * largest)
            over = (got - want).abs() - tol
            assert (over <= 0).all(), f"sequence {b} head {h}: {(over > 0).sum()} of {over.numel()} off, by {over.max():.3g}"
            if weights:
                want = p.sum(0)
                tol = want * (2 * delta.max() + (n + m * group + 16) * 2.0 ** -23) + 2.0 ** -23 * (w0[b, h, :n] + want)
                diff = (w[b, h, :n].double() - w0[b, h, :n].double() - want).abs()
                assert (diff <= tol).all(), f"weights of sequence {b} head {h}: {(diff > tol).sum()} off, by {diff.max():.3g}"
        if weights:
            assert torch.equal(w[b, :, n:], w0[b, :, n:])
    after = (cache.k, cache.k_scales, cache.v, cache.v_scales, cache.page_table, cache.lengths)
    assert all(torch.equal(x, y) for x, y in zip(before, after))


def _queries(rng, shape, dtype, lengths):
    q = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * 1.5).to(dtype).to(DEV)
    return q, [min(shape[1], n) for n in lengths]


def _ragged(rng, batch, top, fixed):
    return (list(fixed) + [int(x) for x in rng.integers(1, top, max(0, batch - len(fixed)))])[:batch]


# one cut of up to 266 pages; one tile of rows and two; with weights
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group,queries,dim,weights,spread", [(8, 1, 64, True, 0), (8, 3, 64, True, 0), (4, 1, 128, False, 20),
                                                              (6, 5, 128, False, 0), (2, 2, 256, False, 20)])
def test_few_rows_of_long_sequences(group, queries, dim, weights, spread, dtype):
    rng = np.random.default_rng(group * 10 + queries)
    lengths = _ragged(rng, 64, 17000, [17000, 16384, 16385, 16383, 16449, 1, 0, 64 * 257])
    cache = _cache(rng, lengths, 8, dim, absent=(3, 255, 256, 261), spread=spread)
    q, lens = _queries(rng, (64, queries, 8 * group, dim), dtype, lengths)
    _check(cache, q, lens, weights)


# two cuts of 258 pages
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,queries", [(64, 1), (128, 4), (256, 1)])
def test_few_rows_of_two_long_cuts(dim, queries, dtype):
    rng = np.random.default_rng(dim)
    lengths = _ragged(rng, 32, 33000, [33000, 16512, 16513, 16511, 32960])
    cache = _cache(rng, lengths, 8, dim, absent=(256, 258, 500))
    q, lens = _queries(rng, (32, queries, 32, dim), dtype, lengths)
    _check(cache, q, lens, False)


# sixteen tiles of rows for 48 heads: sequences are turned by one every 5 1/3 tiles; up to 80 pages
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,weights,spread", [(64, True, 0), (128, False, 0), (128, False, 20), (256, False, 0)])
def test_prompts_of_many_tiles(dim, weights, spread, dtype):
    rng = np.random.default_rng(dim + spread)
    lengths = [5100, 1030, 4096]
    cache = _cache(rng, lengths, 16, dim, absent=(2, 63, 64, 70), spread=spread)
    q, lens = _queries(rng, (3, 1024, 32, dim), dtype, lengths)
    _check(cache, q, lens, weights)


def test_prompts_with_weights_in_many_shares():
    """Weights of prompts whose rows outnumber the keys' groups of a wave."""
    rng = np.random.default_rng(5)
    cache = _cache(rng, [2100, 700], 2, 128)
    q, lens = _queries(rng, (2, 2000, 16, 128), BF16, [2100, 700])
    _check(cache, q, lens, True)


# four cuts of 67 pages
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompts_over_long_caches(dim, dtype):
    rng = np.random.default_rng(dim + 1)
    lengths = [17000, 4288, 4289, 8577, 60, 49, 12865, 16999]
    cache = _cache(rng, lengths, 8, dim, absent=(64, 66, 67, 134, 265))
    q, lens = _queries(rng, (8, 50, 32, dim), dtype, lengths)
    _check(cache, q, lens, False)
