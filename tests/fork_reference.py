"""Plain implementations on the CPU of the serving calls around forked sequences, written from include/qar.h alone: page
owners served one sequence after another, head norms and rotations in 64 bits."""
import numpy as np

PAGE = 64


# ---------------------------------------------------------------------------
# owners of pages: tables are lists of lists, refs and lengths lists; all are changed in place


def is_page(p, refs):
    return 0 <= p < len(refs)


def pages_of(n):
    return -(-n // PAGE)


def clamp(n, top):
    return min(max(n, 0), top)


def fork(table, lengths, refs, parents, width):
    """-> (table, lengths) of the new sequences."""
    new, counts = [], []
    for p in parents:
        n = clamp(lengths[p], len(table[0]) * PAGE) if 0 <= p < len(table) else 0
        row = [table[p][w] if w < pages_of(n) and is_page(table[p][w], refs) else -1 for w in range(width)]
        for page in row:
            if page >= 0:
                refs[page] += 1
        new.append(row)
        counts.append(n)
    return new, counts


def free(table, lengths, refs, keep=None):
    for b, row in enumerate(table):
        n = min(clamp(lengths[b], len(row) * PAGE), max(keep[b], 0) if keep is not None else 0)
        for w in range(pages_of(n), len(row)):
            if is_page(row[w], refs):
                refs[row[w]] -= 1
            row[w] = -1
        lengths[b] = n


def reserve(table, lengths, refs, tokens):
    """-> (room, source, target)"""
    rooms, sources, targets = [], [], []
    spare = [p for p in range(len(refs)) if refs[p] <= 0][::-1]        # the lowest last
    for b, row in enumerate(table):
        n = clamp(lengths[b], len(row) * PAGE)
        end = min(n + max(tokens[b], 0), len(row) * PAGE)
        source = target = -1
        room, w = 0, n // PAGE
        stuck = end == n
        if not stuck and n % PAGE:
            if not is_page(row[w], refs):
                stuck = True
            elif refs[row[w]] > 1:
                if spare:
                    source, target = row[w], spare.pop()
                    refs[source] -= 1
                    refs[target], row[w] = 1, target
                else:
                    stuck = True
            if not stuck:
                w += 1
                room = min(end, w * PAGE) - n
        while not stuck and n + room < end:
            if not is_page(row[w], refs):
                if not spare:
                    break
                row[w] = spare.pop()
                refs[row[w]] = 1
            w += 1
            room = min(end, w * PAGE) - n
        rooms.append(room)
        sources.append(source)
        targets.append(target)
    return rooms, sources, targets


def compact(table, refs):
    """-> (source, target), without the -1 behind them"""
    live = sum(r > 0 for r in refs)
    source = [p for p in range(live, len(refs)) if refs[p] > 0]
    target = [p for p in range(live) if refs[p] <= 0]
    place = dict(zip(source, target))
    for s, t in place.items():
        refs[t] = refs[s]
    for p in range(live, len(refs)):
        refs[p] = 0
    for row in table:
        row[:] = [place.get(p, p) for p in row]
    return source, target


# ---------------------------------------------------------------------------
# head norms and rotations


def rotate(x, heads, kv_heads, positions, frequencies, q_gain, k_gain, eps, interleaved):
    """x float64 [batch, tokens, heads + 2 kv_heads, dim], positions [batch, tokens] whole numbers, frequencies binary32
    -> (q, k, v) in 64 bits"""
    pairs = len(frequencies)
    q, k, v = np.split(np.asarray(x, np.float64), [heads, heads + kv_heads], axis=2)
    t = positions[..., None].astype(np.float64) * frequencies.astype(np.float64)     # [batch, tokens, pairs]
    c, s = np.cos(t)[:, :, None], np.sin(t)[:, :, None]
    first = np.arange(pairs) * (2 if interleaved else 1)
    second = first + (1 if interleaved else pairs)
    outs = []
    for y, gain in ((q, q_gain), (k, k_gain)):
        y = y.copy()
        if eps is not None:
            y = y / np.sqrt((y ** 2).mean(3, keepdims=True) + eps)
            if gain is not None:
                y = y * gain.astype(np.float64)
        a, b = y[..., first].copy(), y[..., second].copy()
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
        outs.append(y)
    return outs[0], outs[1], v
