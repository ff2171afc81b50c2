"""Attention behind shared prefixes for groups whose first sequences, or all, are shorter than the prefix: ended and released
(qar_kv8_free), cut back, or never begun (a fork without a parent).  Their tables name none of the prefix's pages any more."""
import numpy as np
import pytest
import serve_reference as ref
import torch
from test_gpu_kv8 import HEADS, _attention_tolerance, _ints
from test_gpu_kv8_shared import DTYPES, _check, _shared_cache

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64


def _cut(c, kept):
    """The sequences of `kept` {sequence: tokens} cut back as qar_kv8_free does it: entries behind them are -1."""
    for b, n in kept.items():
        c["lengths"][b] = min(c["lengths"][b], n)
        c["page_table"][b, -(-n // PAGE):] = -1


# few rows, many rows, and (1, 130) many rows of own tokens too
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS + [(8, 2, 256)])
@pytest.mark.parametrize("members,queries", [(5, 1), (70, 1), (3, 130)])
@pytest.mark.parametrize("kept", [{0: 0}, {0: 100, 1: 0, 2: 1}])
def test_first_sequences_ended(kept, members, queries, heads, kv_heads, dim, dtype):
    rng = np.random.default_rng(members + dim)
    prefix = 5 * PAGE + 7
    kept = {b: n for b, n in kept.items() if b < members - 1}
    c = _shared_cache(rng, kv_heads, dim, [0, members], [prefix], [prefix + queries + i % 90 for i in range(members)], 9)
    _cut(c, kept)
    _check(c, [0, members], [prefix], queries, heads, dtype, seed=members)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_several_groups(dim, dtype):
    """The first, the last, several and all of a group's sequences ended; the only one that is left is the 66th."""
    rng = np.random.default_rng(dim)
    starts, prefix = [1, 4, 7, 73, 76], [200, 130, 450, 128]
    lengths = [90] + [prefix[g] + 1 + 5 * i for g in range(4) for i in range(starts[g + 1] - starts[g])] + [60]
    c = _shared_cache(rng, 2, dim, starts, prefix, lengths, 14)
    _cut(c, {1: 0, 6: 10, **{b: b % 3 * 70 for b in range(7, 72)}, 73: 0, 74: 0, 75: 0})
    for queries in (1, 9):
        out = _check(c, starts, prefix, queries, 4, dtype, seed=queries)
        assert (out[73:76] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("members", [3, 90])
def test_pages_behind_all_lengths_do_not_matter(members, dim, dtype):
    """All of a group's sequences end before their prefix does.  The pages between were given ahead: their scales are not set,
    here infinite or next to it."""
    rng = np.random.default_rng(members)
    lengths = [70 + i for i in range(members)]
    c = _shared_cache(rng, 2, dim, [0, members], [9 * PAGE], lengths, 10)
    used = c["page_table"][0, :-(-max(lengths) // PAGE)]
    for p, scale in enumerate((np.inf, 3e38, 1e30)):
        page = c["page_table"][0, 8 - p]
        assert page not in used
        c["v_scales"][page] = scale
    _check(c, [0, members], [9 * PAGE], 1, 4, dtype, seed=members)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,heads", [(128, 8), (64, 40)])
def test_beams_that_end(dim, heads, dtype):
    """The library's own calls: beams fork from a prompt, some get no parent, some end and are released; starts and prefix
    stay, eagerly and in a captured call."""
    rng = np.random.default_rng(dim)
    prompt = ref.make_cache(rng, 1, 2, dim, [500], 8, spare=40)
    cache = ref.to_cache(prompt)
    refs = torch.zeros(cache.k.shape[0], dtype=torch.int32, device=DEV)
    refs[cache.page_table[0].long()] = 1
    into = cache.forked(6, 12)
    starts, prefix = _ints(0, 6), _ints(448)
    q = torch.from_numpy(rng.standard_normal((6, 1, heads, dim)).astype(np.float32)).to(dtype)
    qd = q.to(DEV)
    qar.qar_kv8_fork(cache, refs, _ints(-1, 0, 0, 0, 0, 0), into)
    qar.qar_kv8_attention_shared(into, qd, starts, prefix)              # loads the kernels
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = qar.qar_kv8_attention_shared(into, qd, starts, prefix)
    for keep in ([0] + [500] * 5, [0, 0, 130] + [500] * 3, [0, 0, 130, 0, 0, 400], [0] * 6):
        qar.qar_kv8_free(into, refs, _ints(*keep))
        host = {n: getattr(into, n).cpu().numpy() for n in prompt}
        want = ref.attend(host, q.float().numpy(), [1] * 6, dim ** -0.5)
        tol, _ = _attention_tolerance(want, q, dtype, dim, 500 + PAGE)
        got = qar.qar_kv8_attention_shared(into, qd, starts, prefix)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, captured)
        assert (np.abs(got.double().cpu().numpy() - want["out"]) <= tol).all(), keep
