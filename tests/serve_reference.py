"""Plain implementations of the serving calls on the CPU, written from
include/qar.h alone: binary32 where the header defines a binary32 result
(scales, quotients, values), 64 bits for sums and softmax."""
import numpy as np
import torch

PAGE = 64
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


# ---------------------------------------------------------------------------
# microscaled 4-bit


def mx4_quantize(x):
    """x float array [rows, cols] -> (codes uint8 [rows, nb * 16], scale bytes uint8 [rows, nb])."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    p = np.zeros((rows, nb * 32), np.float64)
    p[:, :cols] = x
    p = p.reshape(rows, nb, 32)
    peak = np.abs(p).max(2)
    e = np.where(peak > 0, np.clip(np.frexp(peak)[1] - 3, -126, 125), -3)
    y = np.abs(p) / np.ldexp(1.0, e)[..., None]
    code = np.zeros(y.shape, np.uint8)
    for c in range(1, 8):                      # the nearest value; the even code at a midpoint
        mid = (GRID[c - 1] + GRID[c]) / 2
        code = np.where((y > mid) | ((y == mid) & (c % 2 == 0)), np.uint8(c), code)
    code = code | (np.signbit(p).astype(np.uint8) << 3)
    pair = code.reshape(rows, nb * 16, 2)
    return (pair[..., 0] | pair[..., 1] << 4).astype(np.uint8), (e + 127).astype(np.uint8)


def mx4_values(codes, scales, cols):
    """The 64-bit values [rows, cols]."""
    rows = codes.shape[0]
    code = np.stack((codes & 15, codes >> 4), 2).reshape(rows, -1, 32)
    v = np.concatenate((GRID, -GRID))[code] * np.ldexp(1.0, scales.astype(np.int64) - 127)[..., None]
    return v.reshape(rows, -1)[:, :cols]


# ---------------------------------------------------------------------------
# the cache: a dict of host tensors with the fields of qar.KvCache


def encode(x, scale):
    """int8 codes of binary32 x for binary32 scales that broadcast against it."""
    x, scale = np.asarray(x, np.float32), np.asarray(scale, np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = np.rint(x / scale)
    return np.where(scale > 0, np.clip(q, -127, 127), 0).astype(np.int8)


def make_cache(rng, batch, kv_heads, dim, lengths, width, spare=3, absent=(), ahead=False):
    """A filled cache: scattered pages, garbage behind every sequence's end, NaN scales in pages that no table names.
    `absent`: (sequence, page) entries that point outside the pool.  `ahead`: entries behind a sequence's end name pages that
    were given to it but hold nothing yet."""
    pages = batch * width + spare
    k = rng.integers(-127, 128, (pages, kv_heads, PAGE, dim)).astype(np.int8)
    v = rng.integers(-127, 128, (pages, kv_heads, dim, PAGE)).astype(np.int8)
    ks = (rng.uniform(0.5, 2, (pages, kv_heads)) / 127).astype(np.float32)
    vs = (rng.uniform(0.5, 2, (pages, kv_heads)) / 127).astype(np.float32)
    table = rng.permutation(pages)[:batch * width].reshape(batch, width).astype(np.int32)
    unused = np.ones(pages, bool)
    for b, n in enumerate(lengths):
        used = -(-n // PAGE)
        unused[table[b, :used]] = False
        if not ahead:
            table[b, used:] = -1
    ks[unused], vs[unused] = np.nan, np.nan
    for b, p in absent:
        table[b, p] = [pages, -7, 2 ** 31 - 1, -2 ** 31][(b + p) % 4]
    return {"k": k, "k_scales": ks, "v": v, "v_scales": vs, "page_table": table,
            "lengths": np.array(lengths, np.int32)}


def page_id(c, b, p):
    i = int(c["page_table"][b, p])
    return i if 0 <= i < c["k"].shape[0] else -1


def sequence(c, b, h, which, n):
    """(binary32 values [n, dim] of tokens 0 .. n - 1, which of them are there)"""
    dim = c["k"].shape[3]
    out, there = np.zeros((n, dim), np.float32), np.zeros(n, bool)
    for p in range(-(-n // PAGE)):
        i = page_id(c, b, p)
        if i < 0:
            continue
        codes = c["k"][i, h] if which == "k" else c["v"][i, h].T
        m = min(PAGE, n - p * PAGE)
        out[p * PAGE:p * PAGE + m] = codes[:m].astype(np.float32) * c[which + "_scales"][i, h]
        there[p * PAGE:p * PAGE + m] = True
    return out, there


def append(c, starts, k_new, v_new):
    """Changes c; arrays are binary32 (already exact for bf16 inputs)."""
    batch, tokens, heads, _ = k_new.shape
    for b in range(batch):
        s = int(starts[b])
        if s < 0:
            continue
        for p in range(s // PAGE, -(-(s + tokens) // PAGE)):
            if p >= c["page_table"].shape[1] or page_id(c, b, p) < 0:
                continue
            i, lo, hi = page_id(c, b, p), max(s, p * PAGE), min(s + tokens, (p + 1) * PAGE)
            old = lo - p * PAGE
            for h in range(heads):
                for which, new in (("k", k_new), ("v", v_new)):
                    x = new[b, lo - s:hi - s, h]
                    codes = c[which][i, h] if which == "k" else c[which][i, h].T
                    before = c[which + "_scales"][i, h] if old else np.float32(0)
                    scale = max(before, np.float32(np.abs(x).max()) / np.float32(127))
                    if old and scale > before:
                        codes[:old] = encode(codes[:old].astype(np.float32) * before, scale)
                    codes[old:old + hi - lo] = encode(x, scale)
                    c[which + "_scales"][i, h] = scale


def attend(c, q, q_lens, scale):
    """-> dict of 64-bit results and what error bounds need:
    out, weights, mass (sum of p |v|), peak (largest sum of |q k| of a row), vmax (largest |v| that a row sees)"""
    batch, queries, heads, dim = q.shape
    kv_heads, width = c["k"].shape[1], c["page_table"].shape[1]
    group = heads // kv_heads
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    weights = np.zeros((batch, kv_heads, width * PAGE))
    peak, vmax = np.zeros((batch, queries, heads)), np.zeros((batch, queries, heads))
    for b in range(batch):
        n = min(max(int(c["lengths"][b]), 0), width * PAGE)
        m = min(max(int(q_lens[b]), 0), queries)
        for h in range(kv_heads):
            k, there = sequence(c, b, h, "k", n)
            v, _ = sequence(c, b, h, "v", n)
            k, v = k.astype(np.float64), v.astype(np.float64)
            for i in range(m):
                sees = max(0, n - m + i + 1)
                at = np.nonzero(there[:sees])[0]
                if at.size == 0:
                    continue
                for j in range(h * group, (h + 1) * group):
                    s = scale * (k[at] @ q[b, i, j].astype(np.float64))
                    peak[b, i, j] = abs(scale) * (np.abs(k[at]) @ np.abs(q[b, i, j].astype(np.float64))).max()
                    vmax[b, i, j] = np.abs(v[at]).max()
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[b, i, j], mass[b, i, j] = p @ v[at], p @ np.abs(v[at])
                    weights[b, h, at] += p
    return {"out": out, "weights": weights, "mass": mass, "peak": peak, "vmax": vmax}


def evict(c, into, weights, recent, keep):
    """Changes into -> (kept, moved)"""
    batch, heads = weights.shape[:2]
    width = c["page_table"].shape[1]
    kept = np.full((batch, heads, keep), -1, np.int32)
    moved = np.zeros((batch, heads, keep), np.float32)
    for b in range(batch):
        n = min(max(int(c["lengths"][b]), 0), width * PAGE)
        into["lengths"][b] = min(n, keep)
        for h in range(heads):
            w = weights[b, h, :n]
            last = min(recent, keep) if n > keep else n
            key = np.where(np.isnan(w[:n - last]), np.inf, w[:n - last].astype(np.float64))
            nan = np.isnan(w[:n - last])
            order = np.lexsort((np.arange(n - last), -key, ~nan))
            index = np.sort(np.concatenate((order[:max(0, keep - last)], np.arange(n - last, n)))).astype(int)
            kept[b, h, :index.size], moved[b, h, :index.size] = index, w[index]
            for which in ("k", "v"):
                x, _ = sequence(c, b, h, which, n)
                x = x[index]
                for p in range(-(-index.size // PAGE)):
                    i = page_id(into, b, p)
                    if i < 0:
                        continue
                    page = x[p * PAGE:(p + 1) * PAGE]
                    scale = np.float32(np.abs(page).max()) / np.float32(127)
                    codes = into[which][i, h] if which == "k" else into[which][i, h].T
                    codes[:len(page)] = encode(page, scale)
                    into[which + "_scales"][i, h] = scale
    return kept, moved


# ---------------------------------------------------------------------------
# to and from the device


def to_cache(c, device="cuda:0"):
    from block_wise_int8_amd import qar
    return qar.KvCache(**{name: torch.from_numpy(np.ascontiguousarray(a).copy()).to(device) for name, a in c.items()})


def copy_of(c):
    return {name: a.copy() for name, a in c.items()}


def data(rng, shape, dtype):
    """(device tensor, its exact binary32 values)"""
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
    return t.to("cuda:0"), t.float().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2
