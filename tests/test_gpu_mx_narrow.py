"""Products with few rows of B, whose tiles are short ones, against the float64 oracle: each
side of the border of 193 rows, at heights of A's groups from one row to several tiles,
whole and broken steps, and more tiles than workgroups.  Bars as in ``test_gpu_mx``."""
import numpy as np
import pytest

from helpers import log, to_dev
from oracle import mx
from test_gpu_mx import _bar, _offsets, _operand

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("n", [1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 194])
@pytest.mark.parametrize("K", [256, 300, 1280, 1504])
@pytest.mark.parametrize("spread", [0, 8])
def test_narrow_product(moe, n, K, spread):
    sizes = [257, 0, 128, 129, 288, 1, 300]
    rng = np.random.default_rng(n * 3 + K + spread)
    off, R, G = _offsets(sizes), sum(sizes), len(sizes)
    a_q, a_e, a = _operand(rng, R, K, spread)
    b_q, b_e, b = _operand(rng, G * n, K, spread)
    log(f"moe_grouped_gemm_mxfp4 narrow n={n} K={K} spread={spread}")
    out, _ = moe.moe_grouped_gemm_mxfp4(a_q, a_e, b_q.view(G, n, -1), b_e.view(G, n, -1), to_dev(off), R,
                                        out_dtype=torch.float32, k_dim=K)
    want, mag = mx.grouped_gemm(a, b.reshape(G, n, K), off)
    if spread == 0:
        assert torch.equal(out.cpu(), torch.from_numpy(want).float())
    else:
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= _bar(want, mag, K, "f32"))


@pytest.mark.parametrize("n", [5, 192, 193])
def test_narrow_product_of_more_tiles_than_workgroups(moe, n):
    sizes, K = [34000, 0, 1, 32900], 64
    rng = np.random.default_rng(n)
    off, R, G = _offsets(sizes), sum(sizes), len(sizes)
    a_q, a_e, a = _operand(rng, R, K, 0)
    b_q, b_e, b = _operand(rng, G * n, K, 0)
    assert moe.moe_grouped_gemm_mxfp4_workspace_bytes(G, R, n, K) > 0
    want, _ = mx.grouped_gemm(a, b.reshape(G, n, K), off)
    want = torch.from_numpy(want).float()
    for call in range(2):
        log(f"moe_grouped_gemm_mxfp4 {R} rows n={n}, call {call}")
        out, _ = moe.moe_grouped_gemm_mxfp4(a_q, a_e, b_q.view(G, n, -1), b_e.view(G, n, -1), to_dev(off), R,
                                            out_dtype=torch.float32, k_dim=K)
        assert torch.equal(out.cpu(), want)
