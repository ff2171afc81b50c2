"""The serving calls' workspaces hold all that their kernels read (no GPU)."""
import pytest

from block_wise_int8_amd import qar


@pytest.mark.parametrize("inner", [32, 33, 257, 1000, 5376, 8000])
def test_mx4_linear_few_rows(inner):
    """Up to 64 rows the quantized x lies in tiles of 16 rows, its rows padded to eight blocks; the product is built for one,
    two and four tiles and reads every one of them: 16 bytes of codes and a scale byte for each block."""
    padded = (inner + 255) // 256 * 8
    for rows in range(1, 65):
        if rows <= 16 and inner % 32 == 0:                             # quantized inside the product
            assert qar.lib().qar_mx4_linear_workspace_bytes(rows, inner, 300) == 0
            continue
        tiles = 1 if rows <= 16 else 2 if rows <= 32 else 4
        assert qar.lib().qar_mx4_linear_workspace_bytes(rows, inner, 300) >= tiles * 16 * padded * (16 + 1), rows


@pytest.mark.parametrize("inner", [64, 515, 5376])
def test_mx4_linear_tiles(inner):
    """More rows: codes of the rows themselves (tiles read the last one again), and a scale byte for each block of whole tiles
    of at most 256 rows of x and of the weights."""
    padded = (inner + 255) // 256 * 8
    for rows in (65, 100, 256, 257, 2100):
        for cols in (1, 64, 257, 8200):
            scales = padded * ((rows + 255) // 256 * 256 + (cols + 255) // 256 * 256)
            assert qar.lib().qar_mx4_linear_workspace_bytes(rows, inner, cols) >= rows * padded * 16 + scales
