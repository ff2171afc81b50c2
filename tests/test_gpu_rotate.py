"""Head norms and rotary positions on the GPU against tests/fork_reference.py."""
import fork_reference as ref
import numpy as np
import pytest
import torch

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.bfloat16, torch.float32]


def _frequencies(pairs):
    return (1e4 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)


def _check(x, heads, kv_heads, positions, frequencies, q_gain=None, k_gain=None, eps=None, interleaved=False, out=None):
    """positions int32[batch] or [batch, tokens]; frequencies binary32 (host)."""
    batch, tokens = x.shape[:2]
    dev = [t if t is None else t.to(DEV) for t in (x, q_gain, k_gain)]
    f = torch.from_numpy(frequencies).to(DEV) if len(frequencies) else None
    got = qar.qar_norm_rotate(dev[0], heads, kv_heads, torch.from_numpy(positions).to(DEV), f, q_gain=dev[1], k_gain=dev[2],
                              eps=eps, interleaved=interleaved, out=out)
    each = positions if positions.ndim == 2 else positions[:, None].astype(np.int64) + np.arange(tokens)
    host = [None if t is None else t.double().numpy() for t in (x, q_gain, k_gain)]
    want = ref.rotate(host[0], heads, kv_heads, each, frequencies, host[1], host[2], eps, interleaved)
    # Sizes of what enters a result: the normed pair.  The sum of squares is off by at most 24 roundings, its root by half
    # of those and two more, the normed value by 17 in all; sine and cosine by 2 units of 2^-24 and what 64 bits lose of
    # the angle; two products and a sum: 24 * 2^-24 of the pair's magnitudes, then the result's own rounding.
    plain = ref.rotate(host[0], heads, kv_heads, each, np.zeros(len(frequencies), np.float32), host[1], host[2], eps, interleaved)
    pairs, half = len(frequencies), torch.finfo(x.dtype).eps / 2
    angle = np.abs(each).max() * np.abs(frequencies).max() if pairs else 0
    for i, (g, w, p) in enumerate(zip(got, want, plain)):
        assert g.dtype == x.dtype and g.shape == w.shape
        if i == 2:
            assert torch.equal(g.cpu(), x[:, :, heads + kv_heads:])
            continue
        size = np.abs(p)
        first = np.arange(pairs) * (2 if interleaved else 1)
        second = first + (1 if interleaved else pairs)
        both = size[..., first] + size[..., second]
        size[..., first], size[..., second] = both, both
        tol = size * (24 * 2.0 ** -24 + angle * 2.0 ** -51) + np.abs(w) * half + 1e-37
        diff = np.abs(g.double().cpu().numpy() - w)
        assert (diff <= tol).all(), f"output {i}: {(diff > tol).sum()} of {diff.size} off, worst {(diff / tol).max():.3g} of the tolerance"
    return got


SHAPES = [(1, 1, 1, 1, 64), (3, 5, 4, 2, 128), (2, 33, 16, 8, 256), (70, 1, 32, 8, 128), (1, 1500, 5, 1, 64), (2, 3, 64, 8, 64),
          (1, 7, 40, 40, 128)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("batch,tokens,heads,kv_heads,dim", SHAPES)
def test_shapes(batch, tokens, heads, kv_heads, dim, interleaved, dtype):
    g = torch.Generator().manual_seed(dim + tokens)
    x = (torch.randn((batch, tokens, heads + 2 * kv_heads, dim), generator=g) * 3).to(dtype)
    gains = [(1 + 0.3 * torch.randn(dim, generator=g)).to(dtype) for _ in range(2)]
    positions = np.random.default_rng(1).integers(0, 5000, batch).astype(np.int32)
    _check(x, heads, kv_heads, positions, _frequencies(dim // 2), *gains, eps=1e-6, interleaved=interleaved)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,pairs", [(64, 0), (64, 1), (64, 8), (64, 31), (128, 5), (128, 24), (128, 63), (256, 32), (256, 100),
                                       (256, 127), (256, 120)])
def test_part_of_a_head(dim, pairs, interleaved, dtype):
    """Any number of pairs, a multiple of eight or not; the rest of a head is normed only."""
    g = torch.Generator().manual_seed(pairs)
    x = torch.randn((2, 9, 10, dim), generator=g).to(dtype)
    _check(x, 6, 2, np.array([[7] * 9, list(range(100, 109))], np.int32), _frequencies(pairs), eps=1e-5, interleaved=interleaved)
    _check(x, 6, 2, np.array([0, 12345], np.int32), _frequencies(pairs), interleaved=interleaved)      # no norm


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_gain(dtype):
    x = torch.randn((2, 3, 8, 64), generator=torch.Generator().manual_seed(5)).to(dtype)
    gain = torch.linspace(-2, 2, 64).to(dtype)
    _check(x, 4, 2, np.array([3, 4], np.int32), _frequencies(32), gain, None, eps=0.5)
    _check(x, 4, 2, np.array([3, 4], np.int32), _frequencies(32), None, gain, eps=0.0)


def test_far_and_negative_positions():
    """Angles of a million and of 2^31 positions keep their fraction; a negative position turns the other way."""
    x = torch.randn((7, 2, 6, 128), generator=torch.Generator().manual_seed(6))
    at = np.array([0, 999_983, 16_777_217, 2 ** 31 - 2, -1, -5000, -2 ** 31], np.int32)
    _check(x, 4, 1, at, _frequencies(64), eps=1e-6)
    _check(x, 4, 1, np.stack([at, at[::-1]], 1), _frequencies(64) * np.float32(3.7), interleaved=True)


def test_each_head_for_itself():
    """A NaN, an infinity or an overflowing sum of squares stays in its head; a head of zeros gives zeros; values keep
    whatever they hold."""
    x = torch.randn((1, 4, 8, 64), generator=torch.Generator().manual_seed(7))
    x[0, 0, 1, 3], x[0, 1, 5, 60], x[0, 2, 0, 0], x[0, 3, 2] = float("nan"), float("inf"), 1e30, 0
    x[0, 0, 6, 1], x[0, 0, 7, 2] = float("-inf"), float("nan")
    f = torch.from_numpy(_frequencies(32)).to(DEV)
    at = torch.zeros(1, dtype=torch.int32, device=DEV)
    q, k, v = (t.cpu() for t in qar.qar_norm_rotate(x.to(DEV), 4, 2, at, f, eps=1e-6))
    assert torch.isnan(q[0, 0, 1]).all() and torch.isnan(k[0, 1, 1]).any() and not torch.isfinite(k[0, 1, 1]).all()
    assert (q[0, 2, 0] == 0).all() and (q[0, 3, 2] == 0).all()        # 1e30 squared is infinite: its root divides all away
    assert torch.equal(v.isnan(), x[:, :, 6:].isnan()) and torch.equal(v.nan_to_num(), x[:, :, 6:].nan_to_num())
    clean = x.clone()
    clean[0, 0, 1], clean[0, 1, 5], clean[0, 2, 0] = 1, 1, 1
    qc, kc, _ = (t.cpu() for t in qar.qar_norm_rotate(clean.to(DEV), 4, 2, at, f, eps=1e-6))
    same_q, same_k = torch.ones(4, 4, dtype=torch.bool), torch.ones(4, 2, dtype=torch.bool)
    same_q[0, 1] = same_q[2, 0] = False
    same_k[1, 1] = False
    assert torch.equal(q[0][same_q], qc[0][same_q]) and torch.equal(k[0][same_k], kc[0][same_k])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pairs", [0, 3, 16, 21])
def test_channels_that_are_not_rotated_are_copied(pairs, interleaved, dtype):
    """Bit for bit without a norm: infinities, NaN and negative zeros beside each other."""
    g = torch.Generator().manual_seed(pairs)
    x = torch.randn((2, 3, 6, 64), generator=g).to(dtype)
    x[..., 2 * pairs:][torch.rand(x[..., 2 * pairs:].shape, generator=g) < 0.2] = float("inf")
    x[..., 2 * pairs:][torch.rand(x[..., 2 * pairs:].shape, generator=g) < 0.2] = -0.0
    x[..., 2 * pairs:][torch.rand(x[..., 2 * pairs:].shape, generator=g) < 0.1] = float("nan")
    f = torch.from_numpy(_frequencies(pairs)).to(DEV) if pairs else None
    got = qar.qar_norm_rotate(x.to(DEV), 4, 1, torch.tensor([5, 7], dtype=torch.int32, device=DEV), f, interleaved=interleaved)
    for y, z in zip(got, (x[:, :, :4], x[:, :, 4:5], x[:, :, 5:])):
        assert torch.equal(torch.isnan(y[..., 2 * pairs:].cpu()), torch.isnan(z[..., 2 * pairs:]))
        y, z = (torch.nan_to_num(t[..., 2 * pairs:].cpu(), nan=1.0, posinf=float("inf")) for t in (y, z))
        assert torch.equal(y, z) and torch.equal(torch.signbit(y), torch.signbit(z))
        assert torch.isfinite(got[0][..., :2 * pairs]).all()


def test_outputs_given_and_surroundings_left_alone():
    x = torch.randn((2, 3, 8, 64), generator=torch.Generator().manual_seed(8))
    room = torch.full((3, 4096), 7.0, device=DEV)
    out = tuple(room[i, 64:64 + 6 * n * 64].view(2, 3, n, 64) for i, n in enumerate((4, 2, 2)))
    got = _check(x, 4, 2, np.array([1, 2], np.int32), _frequencies(32), eps=1e-6, out=out)
    assert all(g.data_ptr() == o.data_ptr() for g, o in zip(got, out))
    for i, n in enumerate((4, 2, 2)):
        assert (room[i, :64] == 7).all() and (room[i, 64 + 6 * n * 64:] == 7).all()


def test_nothing_to_do_and_streams():
    at = torch.zeros(2, dtype=torch.int32, device=DEV)
    q, k, v = qar.qar_norm_rotate(torch.empty((2, 0, 8, 64), device=DEV), 4, 2, at, eps=1e-6)
    assert q.shape == (2, 0, 4, 64) and v.shape == (2, 0, 2, 64)
    x = torch.randn((2, 50, 8, 64), device=DEV)
    f = torch.from_numpy(_frequencies(32)).to(DEV)
    want = qar.qar_norm_rotate(x, 4, 2, at, f, eps=1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qar.qar_norm_rotate(x, 4, 2, at, f, eps=1e-6, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph():
    x, at = torch.randn((3, 1, 8, 128), device=DEV), torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
    f = torch.from_numpy(_frequencies(64)).to(DEV)
    qar.qar_norm_rotate(x, 4, 2, at, f, eps=1e-6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = qar.qar_norm_rotate(x, 4, 2, at, f, eps=1e-6)
    for step in range(3):
        x.copy_(torch.randn_like(x))
        at += 1
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, qar.qar_norm_rotate(x, 4, 2, at, f, eps=1e-6))), step
