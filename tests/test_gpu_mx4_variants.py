"""Every form that qar_mx4_linear picks by its sizes, over runs of k that go round its buffers more than once, against
64-bit products of the definition's values (tests/serve_reference.py).

Up to 64 rows: one, two or four tiles of 16 rows, one or two tiles of 16 columns to a workgroup (two from 8,161 columns, from
5,089 for more than 16 rows), x quantized inside (at most 16 rows of whole blocks) or before.  More rows: tiles of 64, 128 or
256, the largest of which there are 256.
"""
import numpy as np
import pytest
import serve_reference as ref
import torch

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _weights(rng, cols, inner):
    """Packed weights with any code, scales 2^-7 .. 2^3 -> (codes, scales, their 64-bit values), on the GPU."""
    nb = (inner + 31) // 32
    codes = torch.from_numpy(rng.integers(0, 256, (cols, nb * 16), dtype=np.uint8)).to(DEV)
    scales = torch.from_numpy(rng.integers(120, 131, (cols, nb), dtype=np.uint8)).to(DEV)
    table = torch.from_numpy(np.concatenate((ref.GRID, -ref.GRID))).to(DEV)
    values = torch.empty((cols, nb, 32), dtype=torch.float64, device=DEV)
    pairs = codes.view(cols, nb, 16).int()
    values[..., 0::2], values[..., 1::2] = table[pairs & 15], table[pairs >> 4]
    values *= torch.exp2(scales.double() - 127)[..., None]
    return codes, scales, values.view(cols, -1)[:, :inner].contiguous()


def _check(rows, inner, cols, dtype, out):
    """Products are exact; binary32 sums of `inner` terms, each addition off by at most 2^-23 of a running sum that the sum of
    magnitudes bounds; one rounding of the result."""
    rng = np.random.default_rng(rows + 31 * inner + 1009 * cols)
    x = torch.from_numpy(rng.standard_normal((rows, inner)).astype(np.float32)).to(dtype)
    codes, scales, wv = _weights(rng, cols, inner)
    xv = torch.from_numpy(ref.mx4_values(*ref.mx4_quantize(x.float().numpy()), inner)).to(DEV)
    need = qar.lib().qar_mx4_linear_workspace_bytes(rows, inner, cols)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device=DEV) if need else None
    y = qar.qar_mx4_linear(x.to(DEV), codes, scales, out_dtype=out, workspace=ws)
    want, size = xv @ wv.T, xv.abs() @ wv.abs().T
    tol = inner * 2.0 ** -23 * size + ref.half_step(out) * want.abs()
    bad = ((y.double() - want).abs() > tol).nonzero()
    assert len(bad) == 0, f"{len(bad)} of {y.numel()}, first at {bad[0].tolist()}"


FEW = [(5, 3840, 8200), (16, 5376, 8161), (1, 32, 8300),               # inside, two tiles of columns
       (16, 5376, 8160),                                               # inside, one
       (7, 1001, 8200), (16, 4097, 8200), (9, 2100, 500),              # one tile of rows
       (17, 1000, 5130), (32, 5376, 5089), (20, 4100, 5088),           # two
       (33, 1000, 5130), (40, 5376, 5130), (48, 257, 5100), (49, 3001, 5130), (64, 5376, 5130), (34, 2000, 33), (48, 4000, 5088)]


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("rows,inner,cols", FEW)
def test_few_rows(rows, inner, cols, dtype, out):
    _check(rows, inner, cols, dtype, out)


# chunks of 256 k through five buffers: one round and its remainders, and more rounds
@pytest.mark.parametrize("inner", [1024, 1280, 1537, 1792, 2300, 2561, 3840, 5377])
@pytest.mark.parametrize("rows,cols", [(100, 300), (300, 11000), (513, 21800)], ids=["64", "128", "256"])
def test_tiles(rows, cols, inner):
    _check(rows, inner, cols, BF16, BF16 if inner % 2 else F32)


@pytest.mark.parametrize("rows,cols", [(90, 130), (257, 16400), (2000, 5376), (700, 22016)], ids=["64", "128", "128s", "256"])
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F32, BF16), (F32, F32)])
def test_tiles_types(rows, cols, dtype, out):
    _check(rows, 1500, cols, dtype, out)


def test_repeats_bit_for_bit():
    """Equal calls, whatever the workspace held, with the tiles of 128 and 256 and 21 chunks."""
    rng = np.random.default_rng(1)
    for rows, cols in ((300, 11000), (513, 21800), (40, 5130)):
        codes, scales, _ = _weights(rng, cols, 5376)
        x, _ = ref.data(rng, (rows, 5376), BF16)
        need = qar.lib().qar_mx4_linear_workspace_bytes(rows, 5376, cols)
        got = [qar.qar_mx4_linear(x, codes, scales, workspace=torch.full((need,), fill, dtype=torch.uint8, device=DEV))
               for fill in (0, 255, 17, 127)]
        assert torch.isfinite(got[0]).all() and all(torch.equal(got[0], y) for y in got)
