"""Head norms and rotary positions of more tokens than one launch may have workgroups."""
import fork_reference as ref
import numpy as np
import pytest
import torch

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("each", [False, True])
def test_more_than_2_to_the_24_tokens(each):
    """Three sequences, each within a launch: equal to their own calls, bit for bit, and to the definition at both sides of
    where one launch ends."""
    batch, tokens, dim = 3, (1 << 24) // 3 + 2, 64
    assert batch * tokens > 1 << 24
    torch.manual_seed(1)
    x = torch.randn((batch, tokens, 3, dim), device=DEV, dtype=torch.bfloat16)
    f = (1e4 ** (-np.arange(32) / 32)).astype(np.float32)
    first = torch.tensor([5, -7, 1000], dtype=torch.int32, device=DEV)
    positions = first[:, None] + torch.arange(tokens, dtype=torch.int32, device=DEV) if each else first
    args = (torch.from_numpy(f).to(DEV), None, None, 1e-6)
    got = qar.qar_norm_rotate(x, 1, 1, positions, *args)
    for b in range(batch):
        own = qar.qar_norm_rotate(x[b:b + 1], 1, 1, positions[b:b + 1].contiguous(), *args)
        for g, o in zip(got, own):
            assert torch.equal(g[b:b + 1], o)
    end = (1 << 24) - 1                                                 # of the first launch, and the call's own end
    for row in (0, end - 1, end, batch * tokens - 1):
        b, t = divmod(row, tokens)
        want = ref.rotate(x[b:b + 1, t:t + 1].double().cpu().numpy(), 1, 1, np.array([[int(first[b]) + t]]), f, None, None, 1e-6, False)
        for g, w in zip(got, want):
            # the result's own rounding; of a pair, whose magnitudes sum to 16 at most, 24 roundings of 2^-24 and the angle's
            tol = torch.finfo(torch.bfloat16).eps / 2 * np.abs(w[0, 0]) + 16 * (24 * 2.0 ** -24 + 2.0 ** -27)
            assert (np.abs(g[b, t].double().cpu().numpy() - w[0, 0]) <= tol).all()
