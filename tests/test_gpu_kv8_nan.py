"""A NaN in a query: its row, and the weights of the tokens that the row sees."""
import numpy as np
import pytest
import serve_reference as ref
import torch

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("queries,heads,n", [(1, 4, 300), (3, 4, 2000), (6, 4, 70), (60, 4, 200), (200, 4, 1500)])
def test_weights(queries, heads, n, dtype):
    """The row of a middle query of one head is NaN; the weights of the tokens that it sees are, of its key head; the others
    are what they are without it, and outputs of the other rows equal."""
    rng = np.random.default_rng(n)
    cache = ref.to_cache(ref.make_cache(rng, 2, 2, 64, [n, n - 7], -(-n // 64) + 1))
    q, _ = ref.data(rng, (2, queries, heads, 64), dtype)
    width = cache.page_table.shape[1] * 64
    clean, weights = torch.zeros((2, 2, width), device="cuda:0"), torch.zeros((2, 2, width), device="cuda:0")
    want = qar.qar_kv8_attention(cache, q, weights=clean)
    i = queries // 2
    q[0, i, 3, 11] = float("nan")
    got = qar.qar_kv8_attention(cache, q, weights=weights)
    assert torch.isnan(got[0, i, 3]).all()
    got[0, i, 3] = want[0, i, 3]
    assert torch.equal(got, want)
    sees = n - queries + i + 1
    assert torch.isnan(weights[0, 1, :sees]).all()
    weights[0, 1, :sees] = clean[0, 1, :sees]
    assert torch.equal(weights, clean)
