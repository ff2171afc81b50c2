"""Many answers to one prompt on libqar: prompts enter a pool of pages once,
every answer forks from its prompt and shares the prompt's pages, attention
reads them once for all answers, and beams fork again as they go.

    python examples/many_answers.py             # on an MI355X

Behind each prompt `answers` sequences generate a token at a time.  Every
`every` tokens the best half of a prompt's answers (by a score that stands for a
model's) goes on twice and the rest is freed; in the end half of the prompts are
freed and the others' pages move to the pool's front.  Each step checks the
attention against a 64-bit softmax over the values that each sequence's pages
hold.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decoder_layer import DecoderLayer, attention_error  # noqa: E402

from block_wise_int8_amd import qar  # noqa: E402


class Answers:
    """Sequences in one pool, grouped by the prompt they answer."""

    def __init__(self, layer, prompts, pages, width):
        self.layer = layer
        self.cache = qar.KvCache.empty(pages, layer.kv_heads, layer.dim, prompts, width)
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.groups = torch.arange(prompts + 1, dtype=torch.int32, device="cuda")
        self.prefix = torch.zeros(prompts, dtype=torch.int32, device="cuda")   # tokens that a prompt's sequences share

    def reserve(self, tokens):
        """Room for `tokens` more tokens of every sequence, in pages that are its own."""
        want = torch.full_like(self.cache.lengths, tokens)
        room, source, target = qar.qar_kv8_reserve(self.cache, self.refs, want)
        qar.qar_kv8_copy(self.cache, source, target)
        assert torch.equal(room, want), "the pool is too small"

    def step(self, x):
        """x [sequences, tokens, hidden] -> the layer's output, the new tokens in the cache."""
        tokens = x.shape[1]
        self.reserve(tokens)
        q, k, v = self.layer.project(x, self.cache.lengths)
        qar.qar_kv8_append(self.cache, self.cache.lengths.clone(), k, v)
        self.cache.lengths += tokens
        attended = qar.qar_kv8_attention_shared(self.cache, q, self.groups, self.prefix)
        self.last = q, attended
        return self.layer.finish(x, attended)

    def fork(self, parents, groups):
        """Sequence b goes on from sequence parents[b]; those that nothing goes on from are freed."""
        into = self.cache.forked(parents.numel())
        qar.qar_kv8_fork(self.cache, self.refs, parents, into)
        qar.qar_kv8_free(self.cache, self.refs)
        self.cache, self.groups = into, groups

    def compact(self):
        """The pages in use get the pool's lowest numbers."""
        source, target = qar.qar_kv8_compact(self.cache, self.refs)
        qar.qar_kv8_copy(self.cache, source, target)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def main(prompts=3, prompt=150, answers=8, generate=40, every=12, seed=1):
    layer = DecoderLayer(hidden=1152, heads=8, kv_heads=2, dim=128)
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = (prompt + generate) // qar.QAR_KV8_PAGE + 2
    a = Answers(layer, prompts, prompts * (prompt // 64 + 1) + 2 * prompts * answers * (generate // 64 + 2), width)

    def hidden_states(rows, tokens):
        return torch.randn((rows, tokens, layer.hidden), generator=g, device="cuda").bfloat16()

    y = a.step(hidden_states(prompts, prompt))
    errors = [attention_error(a.cache, *a.last)]
    parents = torch.arange(prompts, device="cuda").repeat_interleave(answers).to(torch.int32)
    groups = (torch.arange(prompts + 1, device="cuda") * answers).to(torch.int32)
    a.prefix.fill_(prompt)
    a.fork(parents, groups)
    y = y[:, -1:][parents.long()]
    forks = 1
    for token in range(generate):
        noise = 0.1 * hidden_states(prompts * answers, 1)                # what sampling makes of equal states
        y = a.step((torch.nn.functional.normalize(y.float(), dim=2) * layer.hidden ** 0.5).bfloat16() + noise)
        errors.append(attention_error(a.cache, *a.last))
        if token % every == every - 1:
            score = torch.rand((prompts, answers), generator=g, device="cuda")
            best = score.argsort(1, descending=True)[:, :answers // 2].sort(1).values.repeat_interleave(2, 1)
            parents = (best + groups[:-1, None]).flatten().to(torch.int32)
            a.fork(parents, groups)
            y = y[parents.long()]
            forks += 1
    # half of the prompts are answered; what is left moves together
    left = [b for p in range(0, prompts, 2) for b in range(p * answers, (p + 1) * answers)]
    keep = prompts - prompts // 2
    a.fork(_ints(left), groups[:keep + 1].contiguous())
    a.prefix = a.prefix[:keep].contiguous()
    a.compact()
    used = int((a.refs > 0).sum())
    assert (a.refs[used:] == 0).all() and int(a.cache.page_table.max()) < used
    y = a.step((torch.nn.functional.normalize(y[_ints(left).long()].float(), dim=2) * layer.hidden ** 0.5).bfloat16())
    errors.append(attention_error(a.cache, *a.last))
    assert torch.isfinite(y).all()
    qar.qar_kv8_free(a.cache, a.refs)
    return max(errors), forks, used, int(a.refs.abs().sum())


if __name__ == "__main__":
    error, forks, used, owned = main()
    print(f"attention within {error:.2e} of the 64-bit softmax over each sequence's pages, {forks} forks, {used} pages in use "
          f"at the end, {owned} after the last sequence was freed")
