"""Cases that measure libqar's serving operators, and the operators' plain forms.

Five operators of a decoder layer that is served next to the quantized
AllReduce:

  append     new keys and values enter a paged cache held in 8 bits, one
             scale for each page of tokens and head; the tokens are read back
             as the values their codes stand for
  attend     attention over that cache: single tokens, and whole prompts
  evict      a cache keeps its recent tokens and those with the largest
             accumulated attention weight
  quantize   microscaled 4-bit floating point: blocks of 32 E2M1 codes with a
             power-of-two scale, and back to values
  linear     the product of such weights with activations quantized on the way

With ``own`` false ``run`` computes them in elementary torch operations in 32
bits; with ``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one generated token of each of 32 conversations enters the cache
        {"name": "append-token", "op": "append", "batch": 32, "tokens": 1, "kv_heads": 16, "dim": 128,
         "start": 2040, "ragged": True, "dtype": "bf16"},
        # two prompts enter the cache behind a shared prefix that ends inside a page
        {"name": "append-prompt", "op": "append", "batch": 2, "tokens": 8192, "kv_heads": 8, "dim": 256,
         "start": 75, "ragged": True, "dtype": "bf16"},
        # one user, one token, a short conversation: latency
        {"name": "attend-token", "op": "attend", "batch": 1, "queries": 1, "heads": 16, "kv_heads": 8, "dim": 256,
         "length": 1300, "ragged": False, "weights": False, "dtype": "bf16"},
        # few users with long documents
        {"name": "attend-long", "op": "attend", "batch": 8, "queries": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "length": 65535, "ragged": False, "weights": False, "dtype": "bf16"},
        # a busy server's step, lengths all different, the weights summed for a later eviction
        {"name": "attend-batch-weights", "op": "attend", "batch": 64, "queries": 1, "heads": 64, "kv_heads": 8,
         "dim": 64, "length": 8000, "ragged": True, "weights": True, "dtype": "bf16"},
        # two prompts of different length, causal
        {"name": "attend-prompt", "op": "attend", "batch": 2, "queries": 2048, "heads": 32, "kv_heads": 16,
         "dim": 128, "length": 2048, "ragged": True, "weights": False, "dtype": "bf16"},
        # short conversations pass their budget
        {"name": "evict-short", "op": "evict", "batch": 4, "kv_heads": 8, "dim": 128, "length": 1100, "keep": 512,
         "recent": 128, "ragged": True},
        # long documents cut to a quarter
        {"name": "evict-long", "op": "evict", "batch": 8, "kv_heads": 16, "dim": 128, "length": 16384, "keep": 4096,
         "recent": 1000, "ragged": True},
        # one token's hidden state
        {"name": "quantize-token", "op": "quantize", "rows": 1, "cols": 3840, "dtype": "f32"},
        # a prompt's hidden states
        {"name": "quantize-prompt", "op": "quantize", "rows": 8192, "cols": 5376, "dtype": "bf16"},
        # a few tokens of a decoding step through one projection
        {"name": "linear-token", "op": "linear", "rows": 5, "inner": 3840, "cols": 15360, "dtype": "bf16"},
        # a prompt through a wide projection
        {"name": "linear-prompt", "op": "linear", "rows": 8192, "inner": 5376, "cols": 21504, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict", "quantize", "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    heads, kv_heads, dim = rng.choice([(16, 8, 256), (32, 16, 128), (64, 8, 64), (32, 8, 128), (12, 12, 64),
                                       (10, 2, 128), (8, 1, 256)])
    if op == "append":
        tokens = rng.choice([1, 1, _log(rng, 2, 5000)])
        batch = rng.choice([1, _log(rng, 1, max(1, min(128, 16384 // tokens)))])
        return {"op": op, "batch": batch, "tokens": tokens, "kv_heads": kv_heads, "dim": dim,
                "start": _log(rng, 1, 4000) - 1, "ragged": rng.random() < 0.7, "dtype": dtype}
    if op == "attend" and rng.random() < 0.6:
        length = _log(rng, 1, 100000)
        batch = _log(rng, 1, max(1, min(128, 500000 // length)))
        return {"op": op, "batch": batch, "queries": rng.choice([1, 1, 1, 2, 5]), "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "length": length, "ragged": rng.random() < 0.5,
                "weights": rng.random() < 0.3, "dtype": dtype}
    if op == "attend":
        queries = _log(rng, 20, 2500)
        length = queries + rng.choice([0, 0, _log(rng, 1, 6000)])
        return {"op": op, "batch": rng.choice([1, 2, 3]), "queries": queries, "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "length": length, "ragged": rng.random() < 0.5, "weights": rng.random() < 0.2,
                "dtype": dtype}
    if op == "evict":
        length = _log(rng, 100, 30000)
        keep = max(1, int(length * rng.uniform(0.1, 0.9)))
        return {"op": op, "batch": _log(rng, 1, max(1, min(32, 100000 // length))), "kv_heads": kv_heads,
                "dim": dim, "length": length, "keep": keep, "recent": int(keep * rng.uniform(0, 1)),
                "ragged": rng.random() < 0.5}
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": rng.choice([1152, 2880, 3840, 5376, _log(rng, 1, 8000)]),
                "dtype": dtype}
    return {"op": op, "rows": rng.choice([1, _log(rng, 1, 32), _log(rng, 33, 8000)]),
            "inner": rng.choice([1152, 2880, 3840, 5376, _log(rng, 100, 8000)]),
            "cols": rng.choice([1152, 2880, 3840, 5376, _log(rng, 100, 14000)]), "dtype": dtype}


# ----------------------------------------------------------------------------
# inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(case, top, g):
    """int32 lengths: all `top`, or spread between a third of it and all of it, the first `top` itself."""
    n = torch.full((case["batch"],), top, dtype=torch.int32, device="cuda")
    if case["ragged"]:
        part = torch.rand(case["batch"], generator=g, device="cuda") * 0.65 + 0.35
        part[0] = 1.0
        n = (n * part).round().to(torch.int32).clamp(min=min(1, top))
    return n


def _cache(case, lengths, capacity, g, filled=True):
    """A page pool in the cache's layout: keys [pages, heads, PAGE, dim], values [pages, heads, dim, PAGE], a scale
    for each page and head, the sequences' pages scattered over the pool."""
    batch, heads, dim = case["batch"], case["kv_heads"], case["dim"]
    width = max(1, -(-capacity // PAGE))
    pages = batch * width
    pool = {}
    for name, shape in (("k", (pages, heads, PAGE, dim)), ("v", (pages, heads, dim, PAGE))):
        if filled:
            # normal data whose largest magnitude in a page maps to code 127
            codes = torch.empty(shape, dtype=torch.int8, device="cuda")
            peak = 3.6 + 0.4 * torch.rand((pages, heads), generator=g, device="cuda")
            step = max(1, (1 << 27) // (heads * PAGE * dim))
            for i in range(0, pages, step):
                x = torch.randn(codes[i:i + step].shape, generator=g, device="cuda")
                codes[i:i + step] = (x * (127 / peak[i:i + step, :, None, None])).round_().clamp_(-127, 127)
            scales = peak / 127 * torch.exp(0.2 * torch.randn((pages, heads), generator=g, device="cuda"))
        else:
            codes = torch.zeros(shape, dtype=torch.int8, device="cuda")
            scales = torch.zeros((pages, heads), device="cuda")
        pool[name], pool[name + "_scales"] = codes, scales
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).reshape(batch, width)
    used = (lengths[:, None] + PAGE - 1) // PAGE
    pool["page_table"] = torch.where(torch.arange(width, device="cuda")[None] < used, table, -1).to(torch.int32)
    pool["lengths"] = lengths
    return pool


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    state = {"case": case}
    if op == "append":
        before = _lengths(case, case["start"], g)
        lengths = before + case["tokens"]
        state["cache"] = _cache(case, lengths, case["start"] + case["tokens"], g)
        state["starts"] = before
        state["read_starts"] = before // PAGE * PAGE
        shape = (case["batch"], case["tokens"], case["kv_heads"], case["dim"])
        for name in ("k_new", "v_new"):
            x = torch.randn(shape, generator=g, device="cuda")
            x[..., ::31] *= 2                                        # a few channels stand out
            state[name] = x.to(DTYPES[case["dtype"]])
    elif op == "attend":
        lengths = _lengths(case, case["length"], g)
        state["cache"] = _cache(case, lengths, case["length"], g)
        state["q_lens"] = torch.minimum(lengths, torch.full_like(lengths, case["queries"]))
        q = torch.randn((case["batch"], case["queries"], case["heads"], case["dim"]), generator=g, device="cuda")
        state["q"] = (1.5 * q).to(DTYPES[case["dtype"]])
        state["weights"] = None
        if case["weights"]:
            width = state["cache"]["page_table"].shape[1] * PAGE
            state["weights"] = torch.rand((case["batch"], case["kv_heads"], width), generator=g, device="cuda")
    elif op == "evict":
        lengths = _lengths(case, case["length"], g)
        state["cache"] = _cache(case, lengths, case["length"], g)
        state["into"] = _cache(case, torch.full_like(lengths, case["keep"]), case["keep"], g, filled=False)
        state["read_starts"] = torch.zeros_like(lengths)
        width = state["cache"]["page_table"].shape[1] * PAGE
        # few heavy tokens, many light ones, some equal
        w = torch.exp(2 * torch.randn((case["batch"], case["kv_heads"], width), generator=g, device="cuda"))
        state["weights"] = (w * 64).round() / 64
    elif op == "quantize":
        x = torch.randn((case["rows"], case["cols"]), generator=g, device="cuda")
        x *= torch.exp(torch.randn((case["rows"], 1), generator=g, device="cuda"))
        state["x"] = x.to(DTYPES[case["dtype"]])
    else:
        x = torch.randn((case["rows"], case["inner"]), generator=g, device="cuda")
        state["x"] = (x * torch.exp(0.5 * torch.randn((case["rows"], 1), generator=g, device="cuda"))).to(
            DTYPES[case["dtype"]])
        w = torch.randn((case["cols"], case["inner"]), generator=g, device="cuda") * (case["inner"] ** -0.5)
        state["codes"], state["scales"] = _mx4_pack(w)
    return state


# ----------------------------------------------------------------------------
# plain forms


def _encode(x, scale):
    """Codes of x for a scale: the nearest integer of the 32-bit quotient, ties to even, 0 for a scale of 0."""
    q = torch.round(x / torch.where(scale > 0, scale, torch.ones_like(scale))).clamp(-127, 127)
    return torch.where(scale > 0, q, torch.zeros_like(q))


def _as_scale(peak):
    return peak / torch.full_like(peak, 127.0)


def _dense(cache, which):
    """The whole cache as 32-bit values [batch, heads, tokens, dim], zero behind each sequence's length."""
    table = cache["page_table"].clamp(min=0).long()
    x = cache[which][table].float() * cache[which + "_scales"][table][..., None, None]
    if which == "v":
        x = x.transpose(3, 4)
    batch, width, heads, page, dim = x.shape
    x = x.permute(0, 2, 1, 3, 4).reshape(batch, heads, width * page, dim)
    there = torch.arange(width * page, device=x.device) < cache["lengths"][:, None]
    return torch.where(there[:, None, :, None], x, torch.zeros((), device=x.device))


def _read(cache, starts, tokens):
    """Tokens starts .. starts + tokens - 1 of each sequence as [batch, tokens, heads, dim], zero behind its length."""
    at = starts[:, None].long() + torch.arange(tokens, device=starts.device)
    there = at < cache["lengths"][:, None]
    at = torch.where(there, at, torch.zeros_like(at))
    page = cache["page_table"].long().gather(1, at // PAGE).clamp(min=0)
    heads = torch.arange(cache["k"].shape[1], device=starts.device)
    pick = (page[:, :, None], heads[None, None], (at % PAGE)[:, :, None])
    k = cache["k"][pick].float() * cache["k_scales"][pick[:2]][..., None]
    v = cache["v"].transpose(2, 3)[pick].float() * cache["v_scales"][pick[:2]][..., None]
    there = there[:, :, None, None]
    return torch.where(there, k, torch.zeros_like(k)), torch.where(there, v, torch.zeros_like(v))


def _append(cache, starts, k_new, v_new):
    batch, tokens, heads, dim = k_new.shape
    first = starts // PAGE                                           # the first page touched
    count = (tokens + PAGE - 2) // PAGE + 1                          # pages that `tokens` tokens can touch
    index = first[:, None].long() + torch.arange(count, device=starts.device)
    width = cache["page_table"].shape[1]
    page = cache["page_table"].long().gather(1, index.clamp(max=width - 1))
    at = index[:, :, None] * PAGE + torch.arange(PAGE, device=starts.device)   # token positions [batch, count, PAGE]
    row = at - starts[:, None, None]
    new = (row >= 0) & (row < tokens) & (index < width)[:, :, None]
    old = (at < starts[:, None, None])
    row = row.clamp(0, tokens - 1).reshape(batch, -1)
    touched = new.any(2)
    for name, x in (("k", k_new), ("v", v_new)):
        picked = x.float()[torch.arange(batch, device=row.device)[:, None], row]
        x = picked.reshape(batch, count, PAGE, heads, dim).permute(0, 1, 3, 2, 4)    # [batch, count, heads, PAGE, dim]
        mask = new[:, :, None, :, None]
        x = torch.where(mask, x, torch.zeros_like(x))
        safe = page.clamp(min=0)
        before = torch.where(old.any(2)[:, :, None], cache[name + "_scales"][safe], torch.zeros((), device=row.device))
        scale = torch.maximum(before, _as_scale(x.abs().amax((3, 4))))
        codes = cache[name][safe]
        codes = codes.transpose(3, 4) if name == "v" else codes
        kept = torch.where(old[:, :, None, :, None], codes.float(), torch.zeros((), device=row.device))
        again = _encode(kept * before[..., None, None], scale[..., None, None])
        kept = torch.where((scale > before)[..., None, None], again, kept)
        codes = torch.where(mask, _encode(x, scale[..., None, None]), kept).to(torch.int8)
        codes = codes.transpose(3, 4) if name == "v" else codes
        cache[name][page[touched]] = codes[touched]
        cache[name + "_scales"][page[touched]] = scale[touched]


def _attend(cache, q, q_lens, weights):
    batch, queries, heads, dim = q.shape
    k, v = _dense(cache, "k"), _dense(cache, "v")
    kv_heads, tokens = k.shape[1], k.shape[2]
    group = heads // kv_heads
    rows = q.float().reshape(batch, queries, kv_heads, group, dim).permute(0, 2, 1, 3, 4)
    rows = rows.reshape(batch, kv_heads, queries * group, dim)
    s = torch.matmul(rows, k.transpose(2, 3).contiguous()) * (dim ** -0.5)
    i = torch.arange(queries, device=q.device).repeat_interleave(group)
    last = (cache["lengths"] - q_lens)[:, None] + i                  # the last key that a row sees
    last = torch.where(i < q_lens[:, None], last, torch.full_like(last, -1))
    seen = (torch.arange(tokens, device=q.device) <= last[:, None, :, None])
    s = torch.where(seen, s, torch.full((), -math.inf, device=q.device))
    top = s.amax(3, keepdim=True)
    e = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum(3, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    out = torch.matmul(p, v).reshape(batch, kv_heads, queries, group, dim).permute(0, 2, 1, 3, 4)
    if weights is not None:
        weights += p.sum(2)
    return out.reshape(batch, queries, heads, dim).to(q.dtype)


def _evict(cache, into, weights, recent, keep):
    lengths = cache["lengths"]
    tokens = weights.shape[2]
    at = torch.arange(tokens, device=weights.device)
    left = torch.where(lengths > keep, lengths - min(recent, keep), torch.zeros_like(lengths))
    w = torch.where(at < left[:, None, None], weights, torch.full((), math.inf, device=weights.device))
    w = torch.where(at < lengths[:, None, None], w, torch.full((), -math.inf, device=weights.device))
    order = torch.sort(w, dim=2, descending=True, stable=True).indices[:, :, :keep]
    there = torch.arange(order.shape[2], device=w.device) < lengths[:, None, None]
    kept = torch.sort(torch.where(there, order, torch.full_like(order, tokens)), dim=2).values
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[2]), value=tokens)
    there = kept < tokens
    safe = torch.where(there, kept, torch.zeros_like(kept))
    into["lengths"].copy_(torch.clamp(lengths, max=keep))
    width = into["page_table"].shape[1]
    batch, heads = safe.shape[:2]
    page = cache["page_table"].long().gather(1, (safe // PAGE).reshape(batch, -1)).reshape(safe.shape).clamp(min=0)
    pick = (page, torch.arange(heads, device=w.device)[None, :, None], safe % PAGE)
    for name in ("k", "v"):
        codes = cache[name] if name == "k" else cache[name].transpose(2, 3)
        x = codes[pick].float() * cache[name + "_scales"][pick[:2]][..., None]
        x = torch.where(there[..., None], x, torch.zeros_like(x))
        x = torch.nn.functional.pad(x, (0, 0, 0, width * PAGE - keep)).reshape(batch, heads, width, PAGE, -1)
        scale = _as_scale(x.abs().amax((3, 4)))
        codes = _encode(x, scale[..., None, None]).to(torch.int8)
        codes = (codes.transpose(3, 4) if name == "v" else codes).transpose(1, 2)
        into[name][into["page_table"].long()] = codes
        into[name + "_scales"][into["page_table"].long()] = scale.transpose(1, 2)
    moved = torch.where(there, weights.gather(2, safe), torch.zeros((), device=w.device))
    return torch.where(there, kept, torch.full_like(kept, -1)).to(torch.int32), moved


def _power(exponent):
    """2 ** exponent in 32 bits, exactly, for whole exponents from -126 to 127."""
    return ((exponent.to(torch.int32) + 127) << 23).view(torch.float32)


def _mx4(x):
    """x [rows, cols] -> (E2M1 values [rows, blocks, 32], whole exponents [rows, blocks]), the last block padded with 0."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[1] % 32))
    x = x.reshape(x.shape[0], -1, 32)
    exponent = (torch.frexp(x.abs().amax(2)).exponent - 3).clamp(-126, 125)
    y = x * _power(-exponent)[..., None]
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return (torch.round(y / step) * step).clamp(-6, 6), exponent


def _mx4_pack(x):
    """(codes uint8 [rows, blocks * 16], two a byte, the even element low; scales uint8 [rows, blocks], 127 + exponent)"""
    values, exponent = _mx4(x)
    a = values.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code += (values < 0).to(torch.uint8) * 8
    code = code.reshape(x.shape[0], -1, 2)
    return code[..., 0] + code[..., 1] * 16, (exponent + 127).to(torch.uint8)


def _mx4_values(codes, scales):
    """The 32-bit values of packed codes, the padding of the last block among them."""
    code = torch.stack((codes & 15, codes >> 4), 2).reshape(codes.shape[0], -1, 32)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    table = torch.cat((table, -table))
    return (table[code.long()] * _power(scales.int() - 127)[..., None]).reshape(codes.shape[0], -1)


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "append":
        _append(state["cache"], state["starts"], state["k_new"], state["v_new"])
        return _read(state["cache"], state["read_starts"], case["tokens"] + PAGE)
    if op == "attend":
        out = _attend(state["cache"], state["q"], state["q_lens"], state["weights"])
        return out if state["weights"] is None else (out, state["weights"])
    if op == "evict":
        kept, moved = _evict(state["cache"], state["into"], state["weights"], case["recent"], case["keep"])
        return (kept, moved, state["into"]["lengths"], *_read(state["into"], state["read_starts"], case["keep"]))
    x = state["x"]
    values, exponent = _mx4(x)
    values = (values * _power(exponent)[..., None]).reshape(x.shape[0], -1)
    if op == "quantize":
        return values[:, :x.shape[1]].to(x.dtype)
    return torch.matmul(values, _mx4_values(state["codes"], state["scales"]).t()).to(x.dtype)


# ----------------------------------------------------------------------------
# the library's calls


def _own(state):
    from block_wise_int8_amd import qar
    case = state["case"]
    op = case["op"]
    if op == "append":
        cache = qar.KvCache(**state["cache"])
        qar.qar_kv8_append(cache, state["starts"], state["k_new"], state["v_new"])
        return qar.qar_kv8_read(cache, state["read_starts"], case["tokens"] + PAGE, out_dtype=torch.float32)
    if op == "attend":
        out = qar.qar_kv8_attention(qar.KvCache(**state["cache"]), state["q"], q_lens=state["q_lens"],
                                    weights=state["weights"])
        return out if state["weights"] is None else (out, state["weights"])
    if op == "evict":
        into = qar.KvCache(**state["into"])
        kept, moved = qar.qar_kv8_evict(qar.KvCache(**state["cache"]), into, state["weights"], case["recent"],
                                        case["keep"])
        return (kept, moved, into.lengths,
                *qar.qar_kv8_read(into, state["read_starts"], case["keep"], out_dtype=torch.float32))
    x = state["x"]
    if op == "quantize":
        return qar.qar_mx4_dequantize(*qar.qar_mx4_quantize(x), x.shape[1], out_dtype=x.dtype)
    return qar.qar_mx4_linear(x, state["codes"], state["scales"], out_dtype=x.dtype)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------
# what a pass cannot do without


def _mean_length(case, top):
    return max(1, top * 0.675) if case["ragged"] and case["batch"] > 1 else top


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}.get(case.get("dtype"), 4)
    if op == "append":
        new = case["batch"] * case["tokens"] * case["kv_heads"] * case["dim"] * 2
        back = case["batch"] * (case["tokens"] + PAGE // 2) * case["kv_heads"] * case["dim"] * 2
        return {"bytes": new * (size + 1) + back * (1 + 4), "flops": 4 * new + back}
    if op == "attend":
        n = _mean_length(case, case["length"])
        queries = min(case["queries"], n)
        pairs = case["batch"] * case["heads"] * queries * (n - (queries - 1) / 2)
        cache = case["batch"] * case["kv_heads"] * n * (2 * case["dim"] + 8 / PAGE)
        io = 2 * case["batch"] * case["queries"] * case["heads"] * case["dim"] * size
        sums = 8 * case["batch"] * case["kv_heads"] * n if case["weights"] else 0
        return {"bytes": cache + io + sums, "flops": pairs * (4 * case["dim"] + 5)}
    if op == "evict":
        n = _mean_length(case, case["length"])
        keep = min(case["keep"], n) * case["batch"] * case["kv_heads"]
        moved = keep * case["dim"] * 2 * (1 + 1 + 1 + 4)             # read, written, read back, its values
        return {"bytes": 4 * n * case["batch"] * case["kv_heads"] + 8 * keep + moved, "flops": 5 * keep * case["dim"]}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * size + 2 * (0.5 + 1 / 32)), "flops": 5 * n}
    rows, inner, cols = case["rows"], case["inner"], case["cols"]
    return {"bytes": rows * inner * size + cols * inner * (0.5 + 1 / 32) + rows * cols * size,
            "flops": 2 * rows * inner * cols}


# ----------------------------------------------------------------------------
# the definitions in 64 bits.  Where a definition rounds to 32 bits (scales, quotients and values of codes) the 64-bit
# result is rounded there: for one product or quotient of 32-bit numbers that is the 32-bit operation's own result.


def _f32(x):
    return x.float().double()


def _requantize(x):
    """The values that a page [..., PAGE, dim] stands for once it is held in 8 bits."""
    scale = _f32(x.abs().flatten(-2).max(-1).values / 127.0)[..., None, None]
    code = torch.nan_to_num(_f32(x / scale), nan=0.0, posinf=0.0, neginf=0.0).round().clamp(-127, 127)
    return _f32(code * scale), scale


def _pages(cache, which, b, first, last):
    """Pages first .. last - 1 of sequence b as 64-bit values [heads, pages, PAGE, dim], with their scales."""
    ids = cache["page_table"][b, first:last].long()
    x = cache[which][ids].double()
    x = x.transpose(2, 3) if which == "v" else x
    scales = cache[which + "_scales"][ids].double()
    return _f32(x * scales[..., None, None]).transpose(0, 1), scales.t()


def _exact_append(state, case):
    tokens, cache = case["tokens"], state["cache"]
    outs = []
    for which in ("k", "v"):
        out = torch.zeros((case["batch"], tokens + PAGE, case["kv_heads"], case["dim"]), dtype=torch.float64,
                          device="cuda")
        for b in range(case["batch"]):
            start = int(state["starts"][b])
            first, end = start // PAGE, -(-(start + tokens) // PAGE)
            held, scales = _pages(cache, which, b, first, end)
            there = start - first * PAGE                             # tokens that the first page holds already
            held = held.flatten(1, 2)                                # [heads, pages * PAGE, dim]
            x = torch.zeros_like(held)
            x[:, there:there + tokens] = state[which + "_new"][b].double().transpose(0, 1)
            pages = x.unflatten(1, (end - first, PAGE))
            scale = _f32(pages.abs().flatten(2).max(2).values / 127.0)
            if there:
                scale[:, 0] = torch.maximum(scale[:, 0], scales[:, 0])
            s = scale[..., None, None]
            value = _f32(torch.nan_to_num(_f32(pages / s), nan=0.0).round().clamp(-127, 127) * s)
            if there:
                prefix = held[:, :there]
                grown = (scale[:, 0] > scales[:, 0])[:, None, None]
                again = torch.nan_to_num(_f32(prefix / s[:, 0])).round().clamp(-127, 127) * s[:, 0]
                value[:, 0, :there] = torch.where(grown, _f32(again), prefix)
            value = value.flatten(1, 2)[:, :there + tokens].transpose(0, 1)
            out[b, :value.shape[0]] = value[:tokens + PAGE]
        outs.append(out)
    return tuple(outs)


def _exact_attend(state, case):
    cache, q = state["cache"], state["q"].double()
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros_like(q)
    weights = state["weights"].double() if case["weights"] else None
    for b in range(case["batch"]):
        n, m = int(cache["lengths"][b]), int(state["q_lens"][b])
        ids = cache["page_table"][b, :-(-n // PAGE)].long()
        for h in range(case["kv_heads"]):
            k = (cache["k"][ids, h].double() * cache["k_scales"][ids, h].double()[:, None, None]).flatten(0, 1)[:n]
            v = cache["v"][ids, h].double() * cache["v_scales"][ids, h].double()[:, None, None]
            v = v.transpose(1, 2).flatten(0, 1)[:n]
            hidden = torch.ones((m, n), dtype=torch.bool, device="cuda").triu(n - m + 1)
            for j in range(h * group, (h + 1) * group):
                s = (q[b, :m, j] @ k.T / math.sqrt(case["dim"])).masked_fill(hidden, -math.inf)
                p = torch.softmax(s, 1)
                out[b, :m, j] = p @ v
                if weights is not None:
                    weights[b, h, :n] += p.sum(0)
    return out if weights is None else (out, weights)


def _exact_evict(state, case):
    cache, keep, heads = state["cache"], case["keep"], case["kv_heads"]
    kept = np.full((case["batch"], heads, keep), -1, np.int32)
    moved = torch.zeros((case["batch"], heads, keep), dtype=torch.float64, device="cuda")
    lengths = np.minimum(cache["lengths"].cpu().numpy(), keep)
    outs = [torch.zeros((case["batch"], keep, heads, case["dim"]), dtype=torch.float64, device="cuda")
            for _ in range(2)]
    weights = state["weights"].cpu().numpy()
    for b in range(case["batch"]):
        n = int(cache["lengths"][b])
        pages = [_pages(cache, which, b, 0, -(-n // PAGE))[0].flatten(1, 2) for which in ("k", "v")]
        for h in range(heads):
            free = n - min(case["recent"], keep) if n > keep else 0
            heavy = np.lexsort((np.arange(free), -weights[b, h, :free].astype(np.float64)))[:keep - (n - free)]
            index = np.sort(np.concatenate((heavy, np.arange(free, n))))
            kept[b, h, :index.size] = index
            at = torch.from_numpy(index).cuda()
            moved[b, h, :index.size] = state["weights"][b, h, at].double()
            for out, x in zip(outs, pages):
                x = torch.nn.functional.pad(x[h, at], (0, 0, 0, -index.size % PAGE))
                out[b, :index.size, h] = _requantize(x.unflatten(0, (-1, PAGE)))[0].flatten(0, 1)[:index.size]
    return (torch.from_numpy(kept), moved, torch.from_numpy(lengths), *outs)


def _exact_mx4(x):
    """The values of x's blocks of 32: the nearest of E2M1's values times the power of two that puts the block's
    largest magnitude into [4, 8), the one of the even code where two are as near."""
    x = x.double()
    padded = torch.nn.functional.pad(x, (0, -x.shape[1] % 32)).unflatten(1, (-1, 32))
    peak = padded.abs().max(2, keepdim=True).values
    # peak is m * 2 ** e with m in [0.5, 1): 2 ** (e - 3) puts it into [4, 8)
    scale = ((torch.frexp(peak).exponent.long().clamp(min=-120) - 3 + 1023) << 52).view(torch.float64)
    y = (padded / scale).abs()
    value = torch.zeros_like(y)
    grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for code in range(1, 8):
        middle = (grid[code - 1] + grid[code]) / 2
        value = torch.where((y > middle) | ((y == middle) & (code % 2 == 0)), grid[code], value)
    return (torch.copysign(value, padded) * scale).flatten(1)[:, :x.shape[1]]


def _exact_linear(state, case):
    x = _exact_mx4(state["x"])
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                        device="cuda")
    codes = state["codes"].long()
    w = torch.empty((case["cols"], codes.shape[1] * 2), dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = grid[codes % 16], grid[codes // 16]
    w = w.unflatten(1, (-1, 32)) * (state["scales"].long() + (1023 - 127) << 52).view(torch.float64)[..., None]
    return x @ w.flatten(1)[:, :case["inner"]].T


def exact(case, seed):
    state = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "evict": _exact_evict,
            "quantize": lambda s, c: _exact_mx4(s["x"]), "linear": _exact_linear}[case["op"]](state, case)
