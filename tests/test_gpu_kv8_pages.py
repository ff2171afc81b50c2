"""Owners of the cache's pages on the GPU against tests/fork_reference.py, where sequences are served one after another."""
import fork_reference as ref
import numpy as np
import pytest
import serve_reference as serve
import torch

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64
I32 = torch.int32


def _ints(v):
    return torch.tensor(v, dtype=I32, device=DEV)


class Books:
    """A pool with tables on the GPU, and the same as lists."""

    def __init__(self, pages, table, lengths, refs=None, heads=1, dim=64):
        self.cache = qar.KvCache.empty(pages, heads, dim, len(table), len(table[0]), device=DEV)
        self.cache.page_table.copy_(_ints(table))
        self.cache.lengths.copy_(_ints(lengths))
        if refs is None:
            refs = [0] * pages
            for row in table:
                for p in row:
                    if 0 <= p < pages:
                        refs[p] += 1
        self.table, self.lengths, self.host_refs = [list(r) for r in table], list(lengths), list(refs)
        self.refs = _ints(refs)

    def check(self, what):
        assert self.cache.page_table.tolist() == self.table, f"{what}: table"
        assert self.cache.lengths.tolist() == self.lengths, f"{what}: lengths"
        assert self.refs.tolist() == self.host_refs, f"{what}: refs"

    def fork(self, parents, width=None):
        """The forked sequences, sharing this one's refs."""
        into = Books.__new__(Books)
        into.cache = self.cache.forked(len(parents), width)
        into.cache.page_table.fill_(-99)
        into.cache.lengths.fill_(-99)
        into.refs, into.host_refs = self.refs, self.host_refs
        qar.qar_kv8_fork(self.cache, self.refs, _ints(parents), into.cache)
        into.table, into.lengths = ref.fork(self.table, self.lengths, self.host_refs, parents, into.cache.page_table.shape[1])
        into.check("fork")
        self.check("fork leaves the parents alone")
        return into

    def free(self, keep=None):
        qar.qar_kv8_free(self.cache, self.refs, None if keep is None else _ints(keep))
        ref.free(self.table, self.lengths, self.host_refs, keep)
        self.check("free")

    def reserve(self, tokens):
        got = qar.qar_kv8_reserve(self.cache, self.refs, _ints(tokens))
        want = ref.reserve(self.table, self.lengths, self.host_refs, tokens)
        for g, w, what in zip(got, want, ("room", "source", "target")):
            assert g.tolist() == w, what
        self.check("reserve")
        return got

    def compact(self):
        source, target = qar.qar_kv8_compact(self.cache, self.refs)
        ws, wt = ref.compact(self.table, self.host_refs)
        fill = [-1] * (len(self.host_refs) // 2 - len(ws))
        assert source.tolist() == ws + fill and target.tolist() == wt + fill
        self.check("compact")
        return source, target


def _scattered(rng, pages, lengths, width):
    at = iter(rng.permutation(pages).tolist())
    return [[next(at) if w < ref.pages_of(n) else -1 for w in range(width)] for n in lengths]


@pytest.mark.parametrize("pages", [40, 12, 8])
def test_a_beam_search(pages):
    """Forks, cuts and reservations over many steps, tokens one by one, beams that end, pools that are large enough or not."""
    rng = np.random.default_rng(0)
    books = Books(pages, _scattered(rng, pages, [60, 64, 130], 8), [60, 64, 130])
    for step in range(90):
        parents = [int(p) for p in rng.integers(-1 if step % 7 == 0 else 0, len(books.table), 6)]
        new = books.fork(parents)
        books.free()
        room, source, target = new.reserve([1] * 6)
        for b, r in enumerate(room.tolist()):
            new.lengths[b] += r
        new.cache.lengths += room
        books = new


@pytest.mark.parametrize("seed", range(6))
def test_random_calls(seed):
    rng = np.random.default_rng(seed)
    pages = int(rng.integers(1, 400))
    batch, width = int(rng.integers(1, 40)), int(rng.integers(1, 9))
    lengths, left = [], pages
    for _ in range(batch):
        n = int(rng.integers(0, width * PAGE + 1))
        n = n if ref.pages_of(n) <= left else 0
        left -= ref.pages_of(n)
        lengths.append(n)
    books = Books(pages, _scattered(rng, pages, lengths, width), lengths)
    for _ in range(12):
        call = rng.integers(0, 5)
        if call == 0:
            new = books.fork([int(p) for p in rng.integers(-2, len(books.table) + 1, rng.integers(1, 60))],
                             len(books.table[0]) + int(rng.integers(0, 3)))
            books.free()
            books = new
        elif call == 1:
            books.free([int(k) for k in rng.integers(-5, width * PAGE, len(books.table))])
        elif call == 2:
            books.compact()
        else:
            room, _, _ = books.reserve([int(t) for t in rng.choice([-1, 0, 1, 1, 63, 64, 65, 300], len(books.table))])
            take = (room.double() * rng.uniform(0, 1)).ceil().to(I32)
            books.cache.lengths += take
            books.lengths = [n + t for n, t in zip(books.lengths, take.tolist())]


def test_free_what_was_given_ahead():
    """The lengths themselves as what is kept."""
    books = Books(30, [[3, 4, 5, 6], [7, -1, 8, -1], [9, 10, -1, -1]], [70, 64, 0])
    qar.qar_kv8_free(books.cache, books.refs, books.cache.lengths)
    ref.free(books.table, books.lengths, books.host_refs, list(books.lengths))
    books.check("free")
    assert books.table == [[3, 4, -1, -1], [7, -1, -1, -1], [-1] * 4]


def test_reserve_from_one_to_many():
    """Sixty-four go on in one page: all but the last copy it; with other owners besides, the last as well."""
    for others in (0, 1):
        books = Books(300, [[7, 5, 9, -1]], [130])
        new = books.fork([0] * 64)
        if not others:
            books.free()
        _, source, _ = new.reserve([100] * 64)
        assert (source == 9).sum() == 63 + others


@pytest.mark.parametrize("free", range(0, 9))
def test_reserve_when_pages_run_out(free):
    """Every number of free pages below what is wanted: copies, fresh pages, and a last owner whose page is still shared."""
    table = [[0, 1, -1, -1], [2, 3, -1, -1], [0, 1, -1, -1], [2, 3, -1, -1], [0, 1, -1, -1], [4, -1, -1, -1]]
    lengths = [100, 64, 100, 100, 100, 64]
    pages = 5 + free
    books = Books(pages, table, lengths)
    books.reserve([100, 1, 1, 0, 28, 200])


def test_reserve_corner_cases():
    # nothing wanted; tokens below 1; a full table; lengths out of range; absent pages in and behind the last one; pages given ahead
    table = [[0, -1, -1], [1, 2, 3], [1, 2, 3], [-1, -1, -1], [77, -1, -1], [-5, 9, -1], [10, 11, -1], [-1, -1, -1], [13, -1, 14]]
    lengths = [64, 192, 150, 0, 10, 70, 70, -3, 64]
    books = Books(30, table, lengths)
    books.reserve([0, 5, 500, 1, 5, 1, -7, 64, 200])
    books = Books(30, table, lengths)
    books.reserve([1] * 9)
    books = Books(2, [[0], [1]], [1000, 30])                           # longer than its table
    books.reserve([5, 100])
    books = Books(1, [[-1]], [0])
    books.reserve([1])
    books.reserve([1])


def test_reserve_large():
    """More free pages than one look finds, more entries than threads, a long pool whose free pages lie at its end."""
    rng = np.random.default_rng(3)
    pages = 30_000
    refs = [1] * 21_000 + [int(r) for r in rng.integers(0, 2, 9_000)]
    books = Books(pages, [[-1] * 40 for _ in range(300)], [0] * 300, refs)
    books.reserve([int(t) for t in rng.integers(0, 1500, 300)])
    refs = [0] * 20_000
    books = Books(20_000, [[-1] * 7 for _ in range(qar.QAR_KV8_MAX_SEQUENCES)], [0] * qar.QAR_KV8_MAX_SEQUENCES, refs)
    books.reserve([300] * qar.QAR_KV8_MAX_SEQUENCES)
    books.compact()


def test_many_that_share():
    books = Books(5000, [[4999, 17, -1]], [100])
    new = books.fork([0] * qar.QAR_KV8_MAX_SEQUENCES)
    books.free()
    new.reserve([1] * qar.QAR_KV8_MAX_SEQUENCES)


@pytest.mark.parametrize("pages", [1, 2, 3, 64, 8191, 8192, 8193, 20_000])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 1.0])
def test_compact(pages, share):
    rng = np.random.default_rng(pages)
    used = [int(p) for p in np.nonzero(rng.uniform(size=pages) < share)[0]]
    width = 50
    rows = [used[i:i + width] for i in range(0, len(used), width)] or [[-1]]
    table = [r + [-1] * (width - len(r)) for r in rows] + [(used * 50)[:width] or [pages] * width]    # some twice, or none
    table = [(r + [-7] * width)[:width] for r in table]
    Books(pages, table, [0] * len(table)).compact()


def test_compact_counts_below_zero_are_free():
    books = Books(6, [[5, 4, 1]], [0], [-3, 1, 0, -1, 1, 2])
    books.compact()
    assert books.refs.tolist() == [2, 1, 1, 0, 0, 0] or min(books.refs.tolist()) == 0


# ---------------------------------------------------------------------------
# copies


def _pool(rng, pages, heads, dim):
    return serve.make_cache(rng, 1, heads, dim, [pages * PAGE], pages, spare=0)


@pytest.mark.parametrize("heads,dim", [(1, 64), (8, 128), (3, 256), (5, 64), (16, 128)])
def test_copy_within_a_pool(heads, dim):
    rng = np.random.default_rng(heads)
    c = _pool(rng, 30, heads, dim)
    cache = serve.to_cache(c)
    source, target = [3, -1, 29, 7, 7, 30, 4, -9, 2 ** 31 - 1], [10, 11, 0, 8, 15, 1, 30, 2, 9]
    qar.qar_kv8_copy(cache, _ints(source), _ints(target))
    for s, t in zip(source, target):
        if 0 <= s < 30 and 0 <= t < 30:
            for name in ("k", "v", "k_scales", "v_scales"):
                c[name][t] = c[name][s]
    for name in c:
        assert np.array_equal(getattr(cache, name).cpu().numpy(), c[name]), name


def test_copy_between_pools():
    rng = np.random.default_rng(1)
    a, b = _pool(rng, 9, 2, 64), _pool(rng, 500, 2, 64)
    big, small = serve.to_cache(b), serve.to_cache(a)
    source, target = rng.permutation(500)[:9], np.arange(9)[::-1]
    qar.qar_kv8_copy(big, _ints(source.tolist()), _ints(target.tolist()), into=small)
    for name in ("k", "v", "k_scales", "v_scales"):
        assert np.array_equal(getattr(small, name).cpu().numpy()[target], b[name][source]), name
        assert np.array_equal(getattr(big, name).cpu().numpy(), b[name]), name


def test_copy_of_long_lists():
    """More pieces than workgroups, most entries empty."""
    rng = np.random.default_rng(2)
    c = _pool(rng, 1200, 4, 64)
    cache = serve.to_cache(c)
    pages = rng.permutation(1200)
    n = 50_000
    source, target = np.full(n, -1), np.full(n, -1)
    at = rng.permutation(n)[:600]
    source[at], target[at] = pages[:600], pages[600:]
    qar.qar_kv8_copy(cache, _ints(source.tolist()), _ints(target.tolist()))
    for name in ("k", "v", "k_scales", "v_scales"):
        c[name][pages[600:]] = c[name][pages[:600]]
        assert np.array_equal(getattr(cache, name).cpu().numpy(), c[name]), name
    qar.qar_kv8_copy(cache, _ints([]), _ints([]))


def test_far_pages():
    """Pages whose codes lie beyond 4 GiB of the pool's start."""
    pages = 33_000
    cache = qar.KvCache.empty(pages, 8, 256, 1, 2, device=DEV)
    assert cache.k.numel() > 1 << 32
    cache.k[-1], cache.v[-1], cache.k_scales[-1], cache.v_scales[-1] = 3, 4, 5, 6
    qar.qar_kv8_copy(cache, _ints([pages - 1, pages - 1]), _ints([0, pages - 3]))
    for p in (0, pages - 3):
        assert (cache.k[p] == 3).all() and (cache.v[p] == 4).all() and (cache.k_scales[p] == 5).all() and (cache.v_scales[p] == 6).all()
    assert (cache.k[pages - 2] == 0).all() and (cache.k[1] == 0).all()


# ---------------------------------------------------------------------------
# together


def test_forked_sequences_keep_their_tokens():
    """Two go on from one prompt whose last page is partly filled: each reads the prompt and its own tokens."""
    rng = np.random.default_rng(4)
    cache = qar.KvCache.empty(20, 2, 64, 1, 4, device=DEV)
    refs = torch.zeros(20, dtype=I32, device=DEV)
    k = torch.from_numpy(rng.integers(-127, 128, (1, 100, 2, 64)).astype(np.float32)).to(DEV)
    k[:, 0], k[:, 64] = 127, 127                                       # scales of 1: values are kept exactly
    room, _, _ = qar.qar_kv8_reserve(cache, refs, _ints([100]))
    qar.qar_kv8_append(cache, _ints([0]), k, -k)
    cache.lengths += room
    two = cache.forked(2)
    qar.qar_kv8_fork(cache, refs, _ints([0, 0]), two)
    qar.qar_kv8_free(cache, refs)
    room, source, target = qar.qar_kv8_reserve(two, refs, _ints([30, 30]))
    assert room.tolist() == [30, 30]
    qar.qar_kv8_copy(two, source, target)
    more = torch.from_numpy(rng.integers(-127, 128, (2, 30, 2, 64)).astype(np.float32)).to(DEV)
    qar.qar_kv8_append(two, two.lengths.clone(), more, -more)
    two.lengths += room
    got, minus = qar.qar_kv8_read(two, _ints([0, 0]), 130, out_dtype=torch.float32)
    # pages that the new tokens enter behind older ones keep the older ones' scale of 1, or begin with their own
    assert torch.equal(got[:, :100], k.expand(2, -1, -1, -1)) and torch.equal(minus, -got)
    assert torch.equal(got[:, 100:128], more[:, :28])
    assert refs.sum().item() == 1 * 2 + 2 * 2 and refs.tolist()[0] == 2


def test_graph_and_streams():
    """A step that forks, frees, takes pages and copies, captured and replayed between two tables."""
    rng = np.random.default_rng(5)
    books = Books(200, _scattered(rng, 200, [100, 30, 64, 128], 6), [100, 30, 64, 128])
    state = (books.cache.page_table, books.cache.lengths, books.refs)
    first = [t.clone() for t in state]
    parents, tokens = _ints([0, 0, 1, 3]), _ints([1] * 4)
    into = books.cache.forked(4)

    def step():
        qar.qar_kv8_fork(books.cache, books.refs, parents, into)
        qar.qar_kv8_free(books.cache, books.refs)
        room, source, target = qar.qar_kv8_reserve(into, books.refs, tokens)
        qar.qar_kv8_copy(into, source, target)
        into.lengths.add_(room)
        source, target = qar.qar_kv8_compact(into, books.refs)
        qar.qar_kv8_copy(into, source, target)
        books.cache.page_table.copy_(into.page_table)
        books.cache.lengths.copy_(into.lengths)
        return room, source, target

    step()
    for t, f in zip(state, first):
        t.copy_(f)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for t, f in zip(state, first):
        t.copy_(f)
    results = []
    for i in range(5):
        graph.replay()
        torch.cuda.synchronize()
        results.append([t.clone() for t in (*state, *captured)])
    for t, f in zip(state, first):
        t.copy_(f)
    for i in range(5):
        eager = step()
        assert all(torch.equal(a, b) for a, b in zip(results[i], (*state, *eager))), i
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    room, _, _ = qar.qar_kv8_reserve(books.cache, books.refs, tokens, stream=side)
    side.synchronize()
    assert room.tolist() == [1] * 4
