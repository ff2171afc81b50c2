"""The 4-bit product with bias, activation and residual on the GPU, against 64-bit sums and functions."""
import math

import numpy as np
import pytest
import serve_reference as ref
import torch
from test_gpu_mx4_variants import _weights

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
ACTIVATIONS = list(qar.QAR_ACTIVATIONS)
SLOPE = 1.13                                                           # the steepest activation's


def _activation(y, name):
    """64 bits; the tails from erfc and exp, which keep their relative accuracy."""
    if name == "relu":
        return y.clamp(min=0)
    if name == "silu":
        return y / (1 + torch.exp(-y))
    if name == "gelu":
        return 0.5 * y * torch.special.erfc(-y / math.sqrt(2))
    if name == "gelu_tanh":
        return y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def _relative(name, out):
    """The header's bound of an activation."""
    return 0 if name in (None, "relu") else 2.0 ** -16 if out == BF16 else 2.0 ** -21


FLOOR = 90 * 2.0 ** -126                                               # what may become 0


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 40, 70])
@pytest.mark.parametrize("name", ACTIVATIONS)
def test_the_functions(name, rows, out):
    """Products of zeros: the result is the bias's activation.  Every size of number, densely around 0."""
    g = torch.Generator().manual_seed(1)
    y = torch.cat((torch.linspace(-20, 20, 20_001), torch.linspace(-0.01, 0.01, 2_001), torch.randn(20_000, generator=g) * 3,
                   torch.exp2(torch.linspace(-126, 127, 2_000)), -torch.exp2(torch.linspace(-126, 127, 2_000)),
                   torch.linspace(-100, -14, 5_000), torch.tensor([0.0, -0.0, 3.4e38, -3.4e38]))).to(out)
    x = torch.zeros((rows, 64), dtype=BF16, device=DEV)
    codes, scales = qar.qar_mx4_quantize(torch.ones((len(y), 64), device=DEV))
    got = qar.qar_mx4_linear_fused(x, codes, scales, bias=y.to(DEV), activation=name, out_dtype=out).double().cpu()
    want = _activation(y.double(), name)
    want = torch.where(torch.isnan(want), torch.zeros_like(want), want)      # -inf / inf far out
    tol = (_relative(name, out) * (1 + 2.0 ** -8) + ref.half_step(out)) * want.abs() + FLOOR
    bad = ((got - want).abs() > tol).nonzero()
    assert len(bad) == 0, f"{len(bad)}, first at y = {y[bad[0, 1]].item()}: {got[tuple(bad[0])].item()} for {want[bad[0, 1]].item()}"


def _check(rows, inner, cols, dtype, out, bias, name, residual, in_place=False):
    """Binary32 sums as in qar_mx4_linear's test; the bias's addition, the activation (slope and own error), the residual's
    addition and the rounding of the result."""
    rng = np.random.default_rng(rows + 31 * inner + 1009 * cols)
    x = torch.from_numpy(rng.standard_normal((rows, inner)).astype(np.float32)).to(dtype)
    codes, scales, wv = _weights(rng, cols, inner)
    xv = torch.from_numpy(ref.mx4_values(*ref.mx4_quantize(x.float().numpy()), inner)).to(DEV)
    s, size = xv @ wv.T, xv.abs() @ wv.abs().T
    b = torch.from_numpy(rng.standard_normal(cols) * 30).to(out).to(DEV) if bias else None
    r = torch.from_numpy(rng.standard_normal((rows, cols)) * 20).to(out).to(DEV) if residual else None
    z = s + (b.double() if bias else 0)
    act = _activation(z, name)
    act = torch.where(torch.isnan(act), torch.zeros_like(act), act)
    want = act + (r.double() if residual else 0)
    need = qar.lib().qar_mx4_linear_workspace_bytes(rows, inner, cols)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device=DEV) if need else None
    given = r.clone() if in_place else None
    got = qar.qar_mx4_linear_fused(x.to(DEV), codes, scales, bias=b, activation=name, residual=given if in_place else r,
                                   out=given, out_dtype=out, workspace=ws)
    assert got.dtype == out and got.shape == (rows, cols) and (not in_place or got.data_ptr() == given.data_ptr())
    tol = (SLOPE * (inner * 2.0 ** -23 * size + 2.0 ** -24 * z.abs()) + (_relative(name, out) + 2.0 ** -24) * act.abs() +
           2.0 ** -24 * want.abs() + ref.half_step(out) * want.abs() + FLOOR)
    bad = ((got.double() - want).abs() > tol).nonzero()
    assert len(bad) == 0, f"{len(bad)} of {got.numel()}, first at {bad[0].tolist()}"
    return got


SHAPES = [(1, 1, 1), (5, 100, 33), (16, 3840, 64), (16, 257, 8200), (9, 5376, 8170), (17, 129, 100), (32, 2880, 5100),
          (33, 1000, 70), (64, 515, 5257), (65, 64, 64), (100, 1153, 300), (130, 96, 127), (257, 4100, 513), (500, 320, 8200),
          (2100, 320, 8201), (4097, 256, 4097)]


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("rows,inner,cols", SHAPES)
def test_sizes(rows, inner, cols, dtype, out):
    """Every form of the product, each with another mixture."""
    n = SHAPES.index((rows, inner, cols)) + DTYPES.index((dtype, out))
    _check(rows, inner, cols, dtype, out, True, ACTIVATIONS[n % 5], True)
    _check(rows, inner, cols, dtype, out, n % 2 == 0, ACTIVATIONS[(n + 2) % 5], n % 3 == 0, in_place=n % 3 == 0)


DTYPES = [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(3, 50), (40, 70), (300, 200)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("name", ACTIVATIONS)
def test_mixtures(name, bias, residual, rows, cols, out):
    _check(rows, 96, cols, BF16, out, bias, name, residual)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("chunks", range(1, 11))
def test_few_tiles_over_every_number_of_chunks(chunks, out):
    """Few tiles ask for 256 of k three chunks ahead, in a ring of four; whole tiles and ones past the edge."""
    for rows, inner, cols in [(130, 256 * chunks, 200), (128, 256 * chunks - 90, 128)]:
        _check(rows, inner, cols, BF16, out, True, None, True)
        _check(rows, inner, cols, F32, out, False, None, False)


def test_more_tiles_than_two_a_cu():
    """Beside the forms for few tiles: 66 x 33,000 are 1,032 tiles of 64."""
    _check(66, 800, 33_000, BF16, BF16, True, "silu", True)
    _check(66, 800, 33_000, F32, F32, True, None, True)


def test_without_an_epilogue_it_is_the_product():
    rng = np.random.default_rng(2)
    for rows, inner, cols in [(4, 64, 100), (50, 100, 60), (200, 320, 300)]:
        codes, scales, _ = _weights(rng, cols, inner)
        x = torch.from_numpy(rng.standard_normal((rows, inner)).astype(np.float32)).to(DEV)
        assert torch.equal(qar.qar_mx4_linear_fused(x, codes, scales), qar.qar_mx4_linear(x, codes, scales))
        zeros = torch.zeros(cols, device=DEV)
        assert torch.equal(qar.qar_mx4_linear_fused(x, codes, scales, bias=zeros), qar.qar_mx4_linear(x, codes, scales))


def test_in_place_and_surroundings():
    """The residual may be the output; nothing behind it is written, nothing behind the bias is used."""
    _check(7, 77, 45, F32, F32, True, "silu", True, in_place=True)
    _check(70, 77, 45, BF16, BF16, False, None, True, in_place=True)
    rng = np.random.default_rng(3)
    for rows, cols in [(3, 45), (20, 45), (70, 45), (300, 131)]:
        codes, scales, _ = _weights(rng, cols, 77)
        x = torch.from_numpy(rng.standard_normal((rows, 77)).astype(np.float32)).to(DEV)
        flat = torch.full((rows * cols + 64,), 7.0, device=DEV)
        out = flat[:rows * cols].view(rows, cols)
        bias = torch.full((cols + 16,), float("nan"), device=DEV)
        bias[:cols] = 1
        qar.qar_mx4_linear_fused(x, codes, scales, bias=bias[:cols], activation="gelu", residual=out, out=out)
        assert (flat[rows * cols:] == 7).all() and torch.isfinite(out).all()


def test_a_nan_stays_where_it_is():
    x = torch.zeros((20, 64), dtype=F32, device=DEV)
    codes, scales = qar.qar_mx4_quantize(torch.ones((70, 64), device=DEV))
    for name in ACTIVATIONS:
        bias, residual = torch.ones(70, device=DEV), torch.ones((20, 70), device=DEV)
        bias[3], residual[2, 5] = float("nan"), float("nan")
        got = torch.isnan(qar.qar_mx4_linear_fused(x, codes, scales, bias=bias, activation=name, residual=residual)).cpu()
        want = torch.zeros((20, 70), dtype=torch.bool)
        want[:, 3], want[2, 5] = True, True
        assert torch.equal(got, want), name


def test_empty_streams_and_graphs():
    w, s = qar.qar_mx4_quantize(torch.ones((8, 64), device=DEV))
    assert qar.qar_mx4_linear_fused(torch.empty((0, 64), device=DEV), w, s, activation="relu").shape == (0, 8)
    rng = np.random.default_rng(8)
    codes, scales, _ = _weights(rng, 130, 200)
    side = torch.cuda.Stream()
    for rows in (4, 50, 90):
        x, r = (torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)).to(BF16).to(DEV) for n in (200, 130))
        b = torch.ones(130, dtype=BF16, device=DEV)
        args = dict(bias=b, activation="gelu_tanh", residual=r)
        want = qar.qar_mx4_linear_fused(x, codes, scales, **args)
        side.wait_stream(torch.cuda.current_stream())
        y = qar.qar_mx4_linear_fused(x, codes, scales, **args, stream=side)
        side.synchronize()
        assert torch.equal(y, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = qar.qar_mx4_linear_fused(x, codes, scales, **args)
        for _ in range(3):
            x.copy_(torch.randn_like(x))
            r.copy_(torch.randn_like(r))
            want = qar.qar_mx4_linear_fused(x, codes, scales, **args)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
