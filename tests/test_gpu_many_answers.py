"""The example that runs the calls around forked sequences together (examples/many_answers.py)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("kw", [{}, dict(prompts=1, prompt=64, answers=2, generate=5, every=2),
                                dict(prompts=5, prompt=700, answers=4, generate=70, every=20)])
def test_many_answers(kw):
    """Forks, copies, shared attention and compaction: the attention is off by its output's rounding (half a step of bf16) and
    the numerators' (2^-12 each), relative to the largest output; no page is owned by anyone in the end."""
    import many_answers
    error, forks, used, owned = many_answers.main(**kw)
    assert forks == 1 + kw.get("generate", 40) // kw.get("every", 12) and used > 0 and owned == 0
    assert error <= torch.finfo(torch.bfloat16).eps / 2 + 2.0 ** -12 + 2.0 ** -16


def test_a_captured_step():
    """A whole step of forked sequences in one graph (pages taken and copied, norm and rotation, append, attention, products
    with their epilogues), replayed while pages fill and new ones are taken, against the same steps one call at a time."""
    import many_answers
    from block_wise_int8_amd import qar

    def start():
        layer = many_answers.DecoderLayer(hidden=1152, heads=8, kv_heads=2, dim=128)
        a = many_answers.Answers(layer, 2, 60, 5)
        g = torch.Generator(device="cuda").manual_seed(3)
        y = a.step(torch.randn((2, 100, 1152), generator=g, device="cuda").bfloat16())
        parents = torch.tensor([0, 0, 0, 1, 1, 1, 1], dtype=torch.int32, device="cuda")
        a.prefix.fill_(100)
        a.fork(parents, torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda"))
        return layer, a, y[:, -1:][parents.long()].contiguous()

    def step(layer, a, x, ones):
        _, source, target = qar.qar_kv8_reserve(a.cache, a.refs, ones)
        qar.qar_kv8_copy(a.cache, source, target)
        q, k, v = layer.project(x, a.cache.lengths)
        qar.qar_kv8_append(a.cache, a.cache.lengths.clone(), k, v)
        a.cache.lengths += 1
        return layer.finish(x, qar.qar_kv8_attention_shared(a.cache, q, a.groups, a.prefix))

    layer, a, x = start()
    ones = torch.ones(7, dtype=torch.int32, device="cuda")
    want = []
    y = x
    for _ in range(60):
        y = step(layer, a, (y * 0.5).contiguous(), ones)
        want.append(y.clone())
    end = [t.clone() for t in (a.refs, a.cache.page_table, a.cache.lengths)]

    layer, a, x = start()
    held = x.clone()
    state = (a.refs, held, *(getattr(a.cache, name) for name in a.cache.__slots__))
    before = [t.clone() for t in state]
    step(layer, a, held, ones)                                         # warmed up before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.copy_(step(layer, a, (held * 0.5).contiguous(), ones))
    # the step before the capture changed pages, too: the last owner of a page goes on in it
    for t, b in zip(state, before):
        t.copy_(b)
    for i in range(60):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want[i]), i
    assert all(torch.equal(t, e) for t, e in zip((a.refs, a.cache.page_table, a.cache.lengths), end))
