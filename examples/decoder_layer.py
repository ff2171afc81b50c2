"""One decoder layer of a served model on libqar: 4-bit projections, an 8-bit
paged cache, attention that remembers what it attended to, and eviction when a
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
        # two sets of pages in one pool: eviction moves from one to the other
        self.width = capacity // qar.QAR_KV8_PAGE
        self.cache = qar.KvCache.empty(2 * batch * self.width, kv_heads, dim, batch, self.width)
        tables = torch.arange(2 * batch * self.width, dtype=torch.int32, device="cuda").reshape(2, batch, self.width)
        self.cache.page_table.copy_(tables[0])
        self.spare = qar.KvCache(self.cache.k, self.cache.k_scales, self.cache.v, self.cache.v_scales, tables[1].clone(),
                                 torch.zeros_like(self.cache.lengths))
        self.received = torch.zeros((batch, kv_heads, capacity), device="cuda")   # what each token was attended to with
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
        qkv = qar.qar_mx4_linear(x.reshape(batch * tokens, -1), *self.qkv).reshape(batch, tokens, -1, self.dim)
        q, k, v = (t.contiguous() for t in qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=2))
        starts = self.cache.lengths.clone()
        qar.qar_kv8_append(self.cache, starts, k, v)
        self.cache.lengths += tokens
        self.longest += tokens
        attended = qar.qar_kv8_attention(self.cache, q, weights=self.received)
        self.last = q, attended
        x = x + qar.qar_mx4_linear(attended.reshape(batch * tokens, -1), *self.out).reshape(x.shape)
        up = qar.qar_mx4_linear(x.reshape(batch * tokens, -1), *self.up)
        return x + qar.qar_mx4_linear(torch.nn.functional.silu(up), *self.down).reshape(x.shape)

    def attention_error(self):
        """The last step's attention against a 64-bit softmax over the cache's values: the largest difference, relative to
        the largest output."""
        q, attended = self.last
        batch, tokens, heads, _ = q.shape
        n = int(self.cache.lengths.max())
        k, v = (t.double() for t in qar.qar_kv8_read(self.cache, torch.zeros_like(self.cache.lengths), n, torch.float32))
        group = heads // self.kv_heads
        worst = size = 0.0
        for b in range(batch):
            m = int(self.cache.lengths[b])
            hidden = torch.ones((tokens, m), dtype=torch.bool, device="cuda").triu(m - tokens + 1)
            for h in range(heads):
                s = (q[b, :, h].double() @ k[b, :m, h // group].T * self.dim ** -0.5).masked_fill(hidden, -torch.inf)
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
