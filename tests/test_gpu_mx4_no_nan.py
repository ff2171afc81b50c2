"""The 4-bit products of finite numbers are finite: every form of both, over a workspace that holds NaN before the call.  A
result is within its bound or fails, so that a NaN, which is neither above nor below a bound, fails too."""
import numpy as np
import pytest
import serve_reference as ref
import torch
from test_gpu_mx4_fused import ACTIVATIONS, FLOOR, SLOPE, _activation, _relative
from test_gpu_mx4_variants import FEW, _weights

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)]
TILES = [(rows, inner, cols) for rows, cols in [(65, 64), (100, 300), (130, 127), (66, 33_000), (257, 16_400), (2000, 5376), (513, 21_800),
                                                (700, 22_016)] for inner in (256, 700, 1281)]
TILES += [(130, 256 * chunks - 90 * (chunks % 2), 200) for chunks in range(3, 11)]


def _case(rows, inner, cols, dtype):
    rng = np.random.default_rng(rows + 31 * inner + 1009 * cols)
    x = torch.from_numpy(rng.standard_normal((rows, inner)).astype(np.float32)).to(dtype)
    codes, scales, wv = _weights(rng, cols, inner)
    xv = torch.from_numpy(ref.mx4_values(*ref.mx4_quantize(x.float().numpy()), inner)).to(DEV)
    need = qar.lib().qar_mx4_linear_workspace_bytes(rows, inner, cols)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV) if need else None
    return rng, x.to(DEV), codes, scales, xv @ wv.T, xv.abs() @ wv.abs().T, ws


def _within(got, want, tol):
    bad = (~((got.double() - want).abs() <= tol)).nonzero()
    assert len(bad) == 0, f"{len(bad)} of {got.numel()}, first at {bad[0].tolist()}: {got[tuple(bad[0])].item()}"


@pytest.mark.parametrize("rows,inner,cols", FEW + TILES)
def test_every_form(rows, inner, cols):
    """Bounds as in the tests of the two calls: binary32 sums of `inner` terms, the activation's slope and own error, the
    residual's addition and the rounding of the result."""
    n = (FEW + TILES).index((rows, inner, cols))
    for dtype, out in (TYPES[n % 4], TYPES[(n + 1) % 4]):
        rng, x, codes, scales, s, size, ws = _case(rows, inner, cols, dtype)
        sums = inner * 2.0 ** -23 * size
        _within(qar.qar_mx4_linear(x, codes, scales, out_dtype=out, workspace=ws), s, sums + ref.half_step(out) * s.abs())
        for name, residual in ((ACTIVATIONS[n % 5], True), (ACTIVATIONS[(n + 3) % 5], False)):
            b = torch.from_numpy(rng.standard_normal(cols) * 30).to(out).to(DEV)
            r = torch.from_numpy(rng.standard_normal((rows, cols)) * 20).to(out).to(DEV) if residual else None
            z = s + b.double()
            act = _activation(z, name)
            want = act + (r.double() if residual else 0)
            if ws is not None:
                ws.fill_(255)
            got = qar.qar_mx4_linear_fused(x, codes, scales, bias=b, activation=name, residual=r, out_dtype=out, workspace=ws)
            _within(got, want, SLOPE * (sums + 2.0 ** -24 * z.abs()) + (_relative(name, out) + 2.0 ** -24) * act.abs() +
                    2.0 ** -24 * want.abs() + ref.half_step(out) * want.abs() + FLOOR)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 40, 70])
@pytest.mark.parametrize("name", ACTIVATIONS)
def test_finite_arguments(name, rows, out):
    """Every size of number that the type holds: none of the activations of a finite number is infinite or NaN."""
    y = torch.cat((torch.linspace(-200, 200, 4_001), torch.exp2(torch.linspace(-133, 127.9, 4_000)),
                   -torch.exp2(torch.linspace(-133, 127.9, 4_000)), torch.tensor([0.0, -0.0, 3e38, -3e38]))).to(out)
    assert torch.isfinite(y).all()
    x = torch.zeros((rows, 64), dtype=BF16, device=DEV)
    codes, scales = qar.qar_mx4_quantize(torch.ones((len(y), 64), device=DEV))
    got = qar.qar_mx4_linear_fused(x, codes, scales, bias=y.to(DEV), activation=name, out_dtype=out)
    want = _activation(y.double(), name)
    want = torch.where(torch.isnan(want), torch.zeros_like(want), want)      # y / (1 + e^-y): -large / inf
    _within(got, want.to(DEV), (_relative(name, out) * (1 + 2.0 ** -8) + ref.half_step(out)) * want.abs().to(DEV) + FLOOR)
