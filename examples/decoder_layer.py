"""One decoder layer of a served model on libqar: 4-bit projections with their
activations and residuals, normed and rotated queries and keys, an 8-bit paged
cache, attention that remembers what it attended to, and eviction when a
conversation outgrows its budget.

    python examples/decoder_layer.py            # on an MI355X

A prompt enters the cache and is attended to at once; then tokens are generated
one by one.  When the longest sequence reaches the cache's capacity, every head
keeps its recent tokens and the heaviest others in fresh pages and goes on.
Each step checks the attention against a 64-bit softmax over the values that
the cache holds.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_wise_int8_amd import qar  # noqa: E402


class DecoderLayer:
    def __init__(self, hidden=1152, heads=8, kv_heads=4, dim=128, batch=3, capacity=512, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.dim, self.batch = hidden, heads, kv_heads, dim, batch

        def weights(rows, cols):
            return qar.qar_mx4_quantize(torch.randn((rows, cols), generator=g, device="cuda") * cols ** -0.5)
        self.qkv = weights((heads + 2 * kv_heads) * dim, hidden)
        self.out = weights(hidden, heads * dim)
        self.up, self.down = weights(4 * hidden, hidden), weights(hidden, 4 * hidden)
        self.up_bias = (torch.randn(4 * hidden, generator=g, device="cuda") * 0.1).bfloat16()
        self.q_gain, self.k_gain = ((1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).bfloat16() for _ in range(2))
        self.frequencies = 1e4 ** (-torch.arange(dim // 2, device="cuda", dtype=torch.float32) / (dim // 2))
        # two sets of pages in one pool: eviction moves from one to the other
        self.width = capacity // qar.QAR_KV8_PAGE
        self.cache = qar.KvCache.empty(2 * batch * self.width, kv_heads, dim, batch, self.width)
        tables = torch.arange(2 * batch * self.width, dtype=torch.int32, device="cuda").reshape(2, batch, self.width)
        self.cache.page_table.copy_(tables[0])
        self.spare = qar.KvCache(self.cache.k, self.cache.k_scales, self.cache.v, self.cache.v_scales, tables[1].clone(),
                                 torch.zeros_like(self.cache.lengths))
        self.received = torch.zeros((batch, kv_heads, capacity), device="cuda")   # what each token was attended to with
        self.positions = torch.zeros_like(self.cache.lengths)             # tokens seen, kept or not
        self.longest = 0

    def evict(self, keep, recent):
        """Every head keeps `keep` tokens; their weights go with them."""
        _, moved = qar.qar_kv8_evict(self.cache, self.spare, self.received, recent, keep)
        self.cache, self.spare = self.spare, self.cache
        self.received.zero_()
        self.received[:, :, :keep] = moved
        self.longest = min(self.longest, keep)

    def step(self, x):
        """x [batch, tokens, hidden] (bf16) -> the layer's output, the new tokens in the cache."""
        batch, tokens, _ = x.shape
        q, k, v = self.project(x, self.positions)
        starts = self.cache.lengths.clone()
        qar.qar_kv8_append(self.cache, starts, k, v)
        self.cache.lengths += tokens
        self.positions += tokens
        self.longest += tokens
        attended = qar.qar_kv8_attention(self.cache, q, weights=self.received)
        self.last = q, attended
        return self.finish(x, attended)

    def project(self, x, positions):
        """x [batch, tokens, hidden] -> the queries, keys and values of its tokens, which begin at positions[b]."""
        batch, tokens, _ = x.shape
        qkv = qar.qar_mx4_linear(x.reshape(batch * tokens, -1), *self.qkv).reshape(batch, tokens, -1, self.dim)
        return qar.qar_norm_rotate(qkv, self.heads, self.kv_heads, positions, self.frequencies, q_gain=self.q_gain,
                                   k_gain=self.k_gain, eps=1e-6)

    def finish(self, x, attended):
        """The layer behind its attention."""
        rows = x.reshape(-1, self.hidden)
        rows = qar.qar_mx4_linear_fused(attended.reshape(rows.shape[0], -1), *self.out, residual=rows)
        up = qar.qar_mx4_linear_fused(rows, *self.up, bias=self.up_bias, activation="silu")
        return qar.qar_mx4_linear_fused(up, *self.down, residual=rows).reshape(x.shape)

    def attention_error(self):
        """The last step's attention against a 64-bit softmax."""
        return attention_error(self.cache, *self.last)


def attention_error(cache, q, attended):
    """Attention of q over a cache against a 64-bit softmax over the cache's values: the largest difference, relative to the
    largest output."""
    batch, tokens, heads, dim = q.shape
    n = int(cache.lengths.max())
    k, v = (t.double() for t in qar.qar_kv8_read(cache, torch.zeros_like(cache.lengths), n, torch.float32))
    group = heads // k.shape[2]
    worst = size = 0.0
    for b in range(batch):
        m = int(cache.lengths[b])
        hidden = torch.ones((tokens, m), dtype=torch.bool, device="cuda").triu(m - tokens + 1)
        for h in range(heads):
            s = (q[b, :, h].double() @ k[b, :m, h // group].T * dim ** -0.5).masked_fill(hidden, -torch.inf)
            want = torch.softmax(s, 1) @ v[b, :m, h // group]
            worst = max(worst, (attended[b, :, h].double() - want).abs().max().item())
            size = max(size, want.abs().max().item())
    return worst / size


def main(prompt=200, generate=160, capacity=256, keep=128, recent=32, seed=1):
    layer = DecoderLayer(capacity=capacity)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((layer.batch, prompt, layer.hidden), generator=g, device="cuda").bfloat16()
    y = layer.step(x)
    errors, evictions = [layer.attention_error()], 0
    for _ in range(generate):
        if layer.longest == capacity:
            layer.evict(keep, recent)
            evictions += 1
        y = layer.step(torch.nn.functional.normalize(y[:, -1:].float(), dim=2).mul(layer.hidden ** 0.5).bfloat16())
        errors.append(layer.attention_error())
    assert torch.isfinite(y).all()
    return max(errors), evictions


if __name__ == "__main__":
    error, evictions = main()
    print(f"attention within {error:.2e} of the 64-bit softmax over the cache's values, {evictions} evictions")
