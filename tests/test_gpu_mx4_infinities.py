"""The fused 4-bit product where sum + bias is infinite: its activations follow their formulas, whether the infinity comes from
the bias or from a sum that overflows binary32."""
import math

import pytest
import torch

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
INF = math.inf
# of +infinity, of -infinity: there y / (1 + e^-y) and the tanh form are -infinity / infinity
WANT = {None: (INF, -INF), "relu": (INF, 0.0), "silu": (INF, math.nan), "gelu": (INF, 0.0), "gelu_tanh": (INF, math.nan)}
# every form of the product: x quantized inside, one to four tiles of few rows, tiles of 64 (few and many of them), 128, 256
SIZES = [(1, 64, 40), (16, 96, 8200), (20, 100, 70), (60, 64, 70), (70, 300, 130), (66, 64, 33_000), (300, 64, 11_000),
         (4097, 64, 4097)]


def _same(got, want):
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.nan_to_num(got, nan=0.0, posinf=INF, neginf=-INF),
                                                                            torch.nan_to_num(want, nan=0.0, posinf=INF, neginf=-INF))


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows,inner,cols", SIZES)
@pytest.mark.parametrize("name", list(WANT))
def test_infinite_biases(name, rows, inner, cols, out):
    """Products of zeros.  3.4e38 is an infinity in bf16 and none in binary32."""
    x = torch.zeros((rows, inner), dtype=BF16, device=DEV)
    codes, scales = qar.qar_mx4_quantize(torch.ones((cols, inner), device=DEV))
    bias = torch.zeros(cols, dtype=torch.float64)
    bias[1], bias[cols // 2], bias[cols - 1], bias[0] = INF, -INF, INF, 3.4e38
    bias = bias.to(out)
    want = torch.zeros(cols, dtype=torch.float64)                       # every activation of 0 is 0
    want[1], want[cols // 2], want[cols - 1] = WANT[name][0], WANT[name][1], WANT[name][0]
    want[0] = bias[0].double()                                          # far above 0 each is its argument
    for residual in (False, True):
        r = torch.full((rows, cols), 2.0, dtype=out) if residual else None
        got = qar.qar_mx4_linear_fused(x, codes, scales, bias=bias.to(DEV), activation=name, out_dtype=out,
                                       residual=None if r is None else r.to(DEV)).double().cpu()
        total = want + 2 if residual else want
        # 3.4e38 and what activations make of it: exact but for the silu's and the tanh form's quotient
        close = (got[:, 0] - total[0]).abs() <= 2.0 ** -16 * 3.4e38 if math.isfinite(total[0]) else got[:, 0] == total[0]
        assert close.all(), got[0, 0].item()
        assert _same(got[:, 1:], total[1:].expand(rows, cols - 1)), (got[0, 1], got[0, cols // 2], got[0, cols - 1])


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows,inner,cols", SIZES)
@pytest.mark.parametrize("name", list(WANT))
def test_sums_that_overflow(name, rows, inner, cols, out):
    """Finite operands: 2^100 times 2^100 and its negative; the other columns are sums of zeros."""
    x = torch.full((rows, inner), 2.0 ** 100, dtype=F32, device=DEV)
    w = torch.zeros((cols, inner))
    w[1], w[cols - 2] = 2.0 ** 100, -2.0 ** 100
    codes, scales = qar.qar_mx4_quantize(w.to(DEV))
    want = torch.zeros(cols, dtype=torch.float64)
    want[1], want[cols - 2] = WANT[name]
    got = qar.qar_mx4_linear_fused(x, codes, scales, activation=name, out_dtype=out, bias=torch.zeros(cols, dtype=out, device=DEV))
    assert _same(got.double().cpu(), want.expand(rows, cols))
