"""Microscaled 4-bit quantize, dequantize and linear on the GPU against the
definition in 64 bits (tests/serve_reference.py)."""
import numpy as np
import pytest
import serve_reference as ref
import torch

from block_wise_int8_amd import qar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.bfloat16, torch.float32]


def _same(got, want, what):
    got = got.cpu().numpy()
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{what}: {len(bad)} of {want.size} differ, first at {bad[0]}"


def _mixed(rng, rows, cols):
    """Rows of every magnitude, blocks of zeros, signed zeros and one outlier, quotients on every midpoint."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-40, 40, (rows, 1)).astype(np.float64))
    if cols >= 8:
        mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7])       # with a peak in [4, 8)
        x[0, :8] = mid * rng.choice([-1, 1], 8)
    if rows > 2:
        x[1] = 0.0
        x[2] = -0.0
        x[2, cols // 2] = 3e38
    if rows > 4:
        x[3] = rng.standard_normal(cols) * 2.0 ** -130                   # subnormal binary32
        x[4] = rng.standard_normal(cols) * 2.0 ** -146
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (5, 32), (6, 33), (7, 8), (33, 100), (64, 1152), (9, 2884),
                                       (3, 4097), (130, 256)])
def test_quantize_and_back(rows, cols, dtype):
    x = torch.from_numpy(_mixed(np.random.default_rng(rows * 7919 + cols), rows, cols)).to(dtype)
    codes, scales = qar.qar_mx4_quantize(x.to(DEV))
    wc, ws = ref.mx4_quantize(x.float().numpy())
    _same(scales, ws, "scales")
    _same(codes, wc, "codes")
    want = ref.mx4_values(wc, ws, cols)
    for out in DTYPES:
        y = qar.qar_mx4_dequantize(codes, scales, cols, out_dtype=out)
        assert y.dtype == out and y.shape == (rows, cols)
        assert np.array_equal(y.double().cpu().numpy(), want), out


def test_every_bf16_value_at_every_scale_of_its_block():
    """Each finite bf16 value next to peaks up to 2^9 times its magnitude: every quotient the format tells apart."""
    bits = np.arange(1 << 16, dtype=np.uint32)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    x = (bits << 16).view(np.float32)
    for shift in range(0, 10):
        block = np.zeros((x.size, 32), np.float32)
        block[:, 5] = x
        with np.errstate(over="ignore"):
            peak = np.abs(x) * np.float32(2.0 ** shift)
        block[:, 20] = np.where(np.isfinite(peak), peak, 0)
        t = torch.from_numpy(block).to(torch.bfloat16)
        for dtype in DTYPES:
            codes, scales = qar.qar_mx4_quantize(t.to(dtype).to(DEV))
            wc, ws = ref.mx4_quantize(t.float().numpy())
            _same(scales, ws, f"scales, shift {shift}, {dtype}")
            _same(codes, wc, f"codes, shift {shift}, {dtype}")


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8)[:16], (255, 1))
    codes = np.concatenate([codes + 16 * i for i in range(16)], 1).astype(np.uint8)      # 255 rows of 16 blocks
    scales = np.repeat(np.arange(255, dtype=np.uint8)[:, None], 16, 1)
    want = ref.mx4_values(codes, scales, 512)
    for out in DTYPES:
        y = qar.qar_mx4_dequantize(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), 512, out_dtype=out)
        big = np.abs(want) > torch.finfo(out).max
        got = y.double().cpu().numpy()
        assert np.array_equal(got[~big], want[~big]) and np.isinf(got[big]).all()


SHAPES = [(1, 1, 1), (1, 32, 16), (5, 100, 33), (16, 3840, 64), (16, 257, 4098), (17, 129, 100), (32, 2880, 1152),
          (33, 1000, 70), (64, 515, 257), (65, 64, 64), (100, 1153, 300), (130, 96, 127), (257, 4100, 513),
          (2100, 320, 8200), (4097, 256, 4097)]


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                       (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("rows,inner,cols", SHAPES)
def test_linear(rows, inner, cols, dtype, out):
    """Exact products, binary32 sums of `inner` terms (each addition off by at most one unit of 2^-23 of the running sum,
    which the sum of magnitudes bounds), one rounding of the result; the matrix unit may flush each of its partial sums that
    is subnormal."""
    rng = np.random.default_rng(rows + 31 * inner + 1009 * cols)
    x = torch.from_numpy(_mixed(rng, rows, inner) if rows < 64 and rows != 5 else
                         rng.standard_normal((rows, inner)).astype(np.float32)).to(dtype)
    if rows > 2 and rows < 64:
        x[2] = torch.from_numpy(rng.standard_normal(inner).astype(np.float32)).to(dtype)   # no sums beyond binary32
    w = (rng.standard_normal((cols, inner)) * np.exp2(rng.integers(-3, 4, (cols, 1)))).astype(np.float32)
    wc, ws = ref.mx4_quantize(w)
    y = qar.qar_mx4_linear(x.to(DEV), torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV), out_dtype=out)
    assert y.dtype == out and y.shape == (rows, cols)
    xv = torch.from_numpy(ref.mx4_values(*ref.mx4_quantize(x.float().numpy()), inner)).to(DEV)
    wv = torch.from_numpy(ref.mx4_values(wc, ws, inner)).to(DEV)
    want, size = xv @ wv.T, xv.abs() @ wv.T.abs()
    tol = inner * 2.0 ** -23 * size + ref.half_step(out) * want.abs() + (inner / 64 + 2) * 2.0 ** -126
    bad = ((y.double() - want).abs() > tol).nonzero()
    assert len(bad) == 0, f"{len(bad)} of {y.numel()}, first at {bad[0].tolist()}"


def test_linear_needs_no_clean_workspace_and_repeats_bit_for_bit():
    rng = np.random.default_rng(5)
    for rows, inner, cols in [(40, 320, 200), (300, 1000, 520)]:
        x, _ = ref.data(rng, (rows, inner), torch.bfloat16)
        w, _ = ref.data(rng, (cols, inner), torch.float32)
        codes, scales = qar.qar_mx4_quantize(w)
        need = qar.lib().qar_mx4_linear_workspace_bytes(rows, inner, cols)
        got = []
        for fill in (0, 255, 17):
            ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
            got.append(qar.qar_mx4_linear(x, codes, scales, workspace=ws))
        assert torch.isfinite(got[0]).all()
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_outputs_are_not_written_behind_their_end():
    rng = np.random.default_rng(6)
    for rows, inner, cols in [(3, 77, 45), (20, 77, 45), (70, 77, 45), (300, 300, 131)]:
        x, _ = ref.data(rng, (rows, inner), torch.float32)
        w, _ = ref.data(rng, (cols, inner), torch.float32)
        codes, scales = qar.qar_mx4_quantize(w)
        flat = torch.full((rows * cols + 64,), 7.0, device=DEV)
        qar.qar_mx4_linear(x, codes, scales, out=flat[:rows * cols].view(rows, cols))
        assert (flat[rows * cols:] == 7).all()
        nb = (inner + 31) // 32
        c = torch.full((rows * nb * 16 + 64,), 9, dtype=torch.uint8, device=DEV)
        s = torch.full((rows * nb + 64,), 9, dtype=torch.uint8, device=DEV)
        qar.qar_mx4_quantize(x, codes=c[:rows * nb * 16], scales=s[:rows * nb])
        assert (c[rows * nb * 16:] == 9).all() and (s[rows * nb:] == 9).all()
        flat.fill_(7.0)
        if rows * inner <= flat.numel() - 64:
            qar.qar_mx4_dequantize(c[:rows * nb * 16].view(rows, -1), s[:rows * nb], inner, out=flat[:rows * inner].view(rows, inner))
        assert (flat[-64:] == 7).all()


def test_empty_calls():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    codes, scales = qar.qar_mx4_quantize(x)
    assert codes.shape == (0, 32) and scales.shape == (0, 2)
    assert qar.qar_mx4_dequantize(codes, scales, 64).shape == (0, 64)
    w, s = qar.qar_mx4_quantize(torch.ones((8, 64), device=DEV))
    assert qar.qar_mx4_linear(x, w, s).shape == (0, 8)


def test_streams_and_graph_replays():
    """On a stream of its own, and captured: every replay gives the eager result on new inputs."""
    rng = np.random.default_rng(8)
    w, _ = ref.data(rng, (130, 200), torch.float32)
    side = torch.cuda.Stream()
    for rows in (4, 50, 90):
        x, _ = ref.data(rng, (rows, 200), torch.bfloat16)
        codes, scales = qar.qar_mx4_quantize(w)
        need = qar.lib().qar_mx4_linear_workspace_bytes(rows, 200, 130)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
        want = qar.qar_mx4_linear(x, codes, scales)
        side.wait_stream(torch.cuda.current_stream())
        y = torch.empty_like(want)
        qar.qar_mx4_linear(x, codes, scales, out=y, workspace=ws, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qar.qar_mx4_linear(x, codes, scales, out=y, workspace=ws)
        for _ in range(4):
            x.copy_(ref.data(rng, (rows, 200), torch.bfloat16)[0])
            want = qar.qar_mx4_linear(x, codes, scales)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
