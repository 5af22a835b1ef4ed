"""The input gradient in 4-bit blocks against the float64 oracle: streamed and in row tiles,
bf16 and float32 gradients, strided rows, sizes of one row and one column, and the weights
turned from strided matrices.  Bars as in ``test_gpu_mx``."""
import numpy as np
import pytest

from helpers import log, to_dev
from oracle import mx
from test_gpu_mx import KINDS, _bar, _offsets, _strided, _tensor, _want

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("sizes,N,K", [([1], 1, 1), ([1, 0, 2], 7168, 65), ([300, 0, 257, 33], 512, 300),
                                       ([129, 640], 1030, 193), ([288], 1280, 520), ([0, 5, 0], 31, 33)], ids=str)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("strided", [False, True])
def test_input_gradient(moe, sizes, N, K, kind, strided):
    rng = np.random.default_rng(sum(sizes) + N + K)
    off, R, G = _offsets(sizes), sum(sizes), len(sizes)
    w, wv = _tensor(rng.standard_normal((G * N, K)), "bf16")
    dy, dyv = _tensor(rng.standard_normal((R, N)), kind)
    w = w.view(G, N, K)
    if strided:
        w, dy = _strided(w, 3, 1), _strided(dy, 5, 3)
    wt_q, wt_e = moe.mxfp4_quant_32x1(w)
    out = torch.full((R + 2, K), 9.0, dtype=KINDS[kind], device="cuda")
    log(f"moe_grouped_dgrad_mxfp4 {sizes} N={N} K={K} {kind} strided={strided}")
    dx = moe.moe_grouped_dgrad_mxfp4(dy, wt_q, wt_e, to_dev(off), out=out[1:R + 1])
    turned = np.stack([_want(wv[g * N:(g + 1) * N].T)[2] for g in range(G)])
    want, mag = mx.grouped_gemm(_want(dyv)[2], turned, off)
    got = dx.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= _bar(want, mag, N, kind))
    assert (out[0] == 9.0).all() and (out[R + 1] == 9.0).all()
