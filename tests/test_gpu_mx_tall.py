"""Tiles of 257 to 288 rows of the 4-bit product (taken where k is a whole number of steps of
256 columns) against the float64 oracle, with scales that differ from block to block:
every count of steps up to two rounds of the K loop, rows plain, gathered and scaled, NaN
blocks in the rows past 256, and the gated epilogue.  Bars as in ``test_gpu_mx``."""
import numpy as np
import pytest

from helpers import log, to_dev
from oracle import mx
from test_gpu_mx import _bar, _check_h, _offsets, _operand

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}
STEPS = [1, 2, 3, 4, 5, 6, 7, 8, 9]


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


def _case(sizes, n, K, spread, a_rows=None):
    rng = np.random.default_rng(sum(sizes) + n + K + spread)
    off, R, G = _offsets(sizes), sum(sizes), len(sizes)
    a_q, a_e, a = _operand(rng, R if a_rows is None else a_rows, K, spread)
    b_q, b_e, b = _operand(rng, G * n, K, spread)
    return rng, off, R, (a_q, a_e), (b_q.view(G, n, -1), b_e.view(G, n, -1)), a, b.reshape(G, n, K)


@pytest.mark.parametrize("sizes", [[257], [288, 0, 257], [270, 575]], ids=str)
@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_plain(moe, sizes, steps, kind):
    n, K = 300, 256 * steps
    _, off, R, A, B, a, b = _case(sizes, n, K, 8)
    log(f"moe_grouped_gemm_mxfp4 tall {sizes} K={K} {kind}")
    out, _ = moe.moe_grouped_gemm_mxfp4(*A, *B, to_dev(off), R, out_dtype=KINDS[kind])
    want, mag = mx.grouped_gemm(a, b, off)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= _bar(want, mag, K, kind))


@pytest.mark.parametrize("sizes", [[288], [257, 3, 281]], ids=str)
@pytest.mark.parametrize("steps", STEPS)
def test_gathered_and_scaled(moe, sizes, steps):
    """Rows gathered from fewer (indices outside are clamped), scaled per row."""
    n, K, T = 264, 256 * steps, 101
    rng, off, R, A, B, a, b = _case(sizes, n, K, 8, T)
    index = rng.integers(0, T, R).astype(np.int32)
    index[0], index[-1] = -5, T + 9
    scale = rng.standard_normal(R).astype(np.float32)
    log(f"moe_grouped_gemm_mxfp4 tall, gathered {sizes} K={K}")
    out, _ = moe.moe_grouped_gemm_mxfp4(*A, *B, to_dev(off), R, a_row_index=to_dev(index),
                                        row_scale=to_dev(scale), out_dtype=torch.float32)
    want, mag = mx.grouped_gemm(a, b, off, np.clip(index, 0, T - 1), scale.astype(np.float64))
    bar = _bar(want, mag, K, "f32") + 2.0 ** -24 * np.abs(want)         # the scale's own rounding
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bar)


@pytest.mark.parametrize("steps", [1, 4, 7])
@pytest.mark.parametrize("gathered", [False, True])
def test_nan_blocks_in_the_last_rows(moe, steps, gathered):
    """A NaN block in a row past 256 and in the last row: NaN there, and nowhere else."""
    sizes, n, K = [288], 256, 256 * steps
    _, off, R, (a_q, a_e), B, a, b = _case(sizes, n, K, 0)
    bad, index = [260, 287], None
    source = np.arange(R)[::-1].copy() if gathered else np.arange(R)
    a_e[source[260], 0] = 255
    # the last block's byte, where a row of scales holds one that is there
    a_e[source[287], -1 if K % 512 == 0 else 0] = 255
    if gathered:
        index, a = to_dev(source.astype(np.int32)), a[source]
    log(f"moe_grouped_gemm_mxfp4 tall with NaN rows K={K} gathered={gathered}")
    out, _ = moe.moe_grouped_gemm_mxfp4(a_q, a_e, *B, to_dev(off), R, a_row_index=index, out_dtype=torch.float32)
    want, _ = mx.grouped_gemm(a, b, off)
    out = out.cpu().numpy()
    assert np.isnan(out[bad]).all()
    keep = np.setdiff1d(np.arange(R), bad)
    assert np.array_equal(out[keep], want[keep].astype(np.float32))


@pytest.mark.parametrize("sizes", [[288], [257, 545]], ids=str)
@pytest.mark.parametrize("steps", [1, 2, 4, 5, 7])
@pytest.mark.parametrize("gathered", [False, True])
def test_gated(moe, sizes, steps, gathered):
    I, K = 384, 256 * steps
    T = 101 if gathered else None
    rng, off, R, A, (b_q, b_e), a, b = _case(sizes, 2 * I, K, 2, T)
    # products of a few units in magnitude, as the activation sees them
    lower = int(np.round(np.log2(np.sqrt(K) * 12)))
    b_e, b = b_e - lower, b * 2.0 ** -lower
    index = rng.integers(0, T, R).astype(np.int32) if gathered else None
    log(f"moe_grouped_gemm_mxfp4 tall, gated {sizes} K={K} gathered={gathered}")
    q, e = moe.moe_grouped_gemm_mxfp4(*A, b_q, b_e, to_dev(off), R, moe.MOE_EPI_SWIGLU_MXFP4,
                                      a_row_index=None if index is None else to_dev(index))
    C, mag = mx.grouped_gemm(a, b, off, index)
    h = mx.gated(C)
    pair = lambda v: [v.reshape(R, -1, 2, 128)[:, :, i].reshape(R, I) for i in (0, 1)]   # noqa: E731
    (g, u), (dg, du) = pair(C), pair(((K + 127) // 128 * 4) * 2.0 ** -24 * mag)
    silu = g / (1 + np.exp(-g))
    tol = 1.1 * np.abs(u) * dg + np.abs(silu) * du + (16 + 2 * np.abs(g)) * 2.0 ** -24 * np.abs(h)
    q, e = q.cpu().numpy(), e.cpu().numpy()
    assert _check_h(q, e, h, tol) <= 1e-3
    blocks = I // 32
    absent = [at // 16 * 16 + 4 * (at % 4) + at % 16 // 4 for at in range(blocks, 16)]
    assert (e[:, absent] == 127).all()
