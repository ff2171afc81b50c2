"""What the roundings that attention chooses can do: binary16 terms on the CPU, and rows of few keys, whose few numerators
carry the whole output, on the GPU."""
import numpy as np
import pytest
import torch

from block_wise_int8_amd import qar


def _values(lo, hi, seed):
    """Binary32 values over [2^lo, 2^hi), those next to binary16's midpoints among them."""
    rng = np.random.default_rng(seed)
    x = np.exp2(rng.uniform(lo, hi, 1 << 18))
    mid = (1 + (2 * np.arange(1024) + 1) * 2.0 ** -11)[None] * np.exp2(np.arange(lo, hi))[:, None]
    near = (mid.reshape(-1)[:, None] * (1 + np.array([-1, 0, 1]) * 2.0 ** -22)).reshape(-1)
    return np.concatenate((x, near)).astype(np.float32)


def test_one_term_is_off_by_half_a_step():
    """2^-11 of the value at most, and more than 2^-12 of it where the significand is small."""
    x = _values(-14, 15, 0)
    off = np.abs(x.astype(np.float64) - x.astype(np.float16).astype(np.float64)) / x
    assert off.max() <= 2.0 ** -11 == torch.finfo(torch.float16).eps / 2
    assert off.max() > 1.99 * 2.0 ** -12


def test_two_terms():
    """2^-23 of the value, or 2^-25 where the second term is subnormal."""
    x = _values(-24, 15, 1)
    hi = x.astype(np.float16)
    lo = (x - hi.astype(np.float32)).astype(np.float16)
    off = np.abs(x.astype(np.float64) - hi.astype(np.float64) - lo.astype(np.float64))
    assert (off <= np.maximum(2.0 ** -23 * x.astype(np.float64), 2.0 ** -25)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("queries,heads,dim", [(1, 8, 64), (37, 8, 64), (50, 8, 128), (20, 4, 256)])
def test_rows_of_few_keys(queries, heads, dim, dtype):
    """Scores: dim exact products (binary32 queries off by 2^-23 of an element) and a few roundings, (dim + 8) 2^-23 of their
    magnitudes' sum, and 2^-20 for the exponential; the softmax's sum doubles both.  A numerator: 2^-11 (one term), 2^-23 or
    2^-39 of the largest value (two).  Sums: (n + 8) 2^-24.  Then one rounding of the output."""
    dev, batch, n = "cuda:0", 64, 50
    g = torch.Generator(device=dev).manual_seed(dim + queries)
    cache = qar.KvCache.empty(batch, heads, dim, batch, 1)
    cache.page_table.copy_(torch.randperm(batch, generator=g, device=dev).to(torch.int32)[:, None])
    cache.lengths.copy_(torch.randint(1, n + 1, (batch,), generator=g, device=dev))
    for name in ("k", "v"):
        getattr(cache, name).copy_(torch.randint(-127, 128, getattr(cache, name).shape, generator=g, device=dev))
        getattr(cache, name + "_scales").copy_((torch.rand((batch, heads), generator=g, device=dev) + 0.5) / 127)
    lens = torch.clamp(cache.lengths, max=queries)
    q = torch.randn((batch, queries, heads, dim), generator=g, device=dev).to(dtype)
    out = qar.qar_kv8_attention(cache, q, q_lens=lens).double()
    rounding = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -23
    for b in range(batch):
        length, m, i = int(cache.lengths[b]), int(lens[b]), int(cache.page_table[b, 0])
        hidden = torch.ones((m, length), dtype=torch.bool, device=dev).triu(length - m + 1)
        for h in range(heads):
            k = cache.k[i, h, :length].double() * cache.k_scales[i, h].double()
            v = (cache.v[i, h].double() * cache.v_scales[i, h].double()).T[:length].contiguous()
            rows = q[b, :m, h].double()
            p = torch.softmax((rows @ k.T * dim ** -0.5).masked_fill(hidden, -torch.inf), 1)
            want = p @ v
            delta = (dim + 8) * 2.0 ** -23 * dim ** -0.5 * (rows.abs() @ k.abs().T).amax(1) + 2.0 ** -20
            tol = ((2 * delta + rounding + (length + 8) * 2.0 ** -24)[:, None] * (p @ v.abs()) + length * 2.0 ** -39 * v.abs().amax()
                   + torch.finfo(dtype).eps / 2 * want.abs())
            over = (out[b, :m, h] - want).abs() - tol
            assert (over <= 0).all(), f"sequence {b} head {h}: {(over > 0).sum()} of {over.numel()} off, by {over.max():.3g}"
