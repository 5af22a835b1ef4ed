"""Every scale of the 4-bit format: the conversions both ways and the product, bit for bit.

A block's scale byte is set by its largest value; the other values are the grid's points and
midpoints times that scale and their neighbours in the type, so that every byte the quantiser
can give meets every tie and both of its sides."""
import numpy as np
import pytest

import synth
from helpers import log, to_dev
from oracle import mx
from test_gpu_mx import _same_values, _tensor, _want

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

GRID = mx.GRID
POINTS = np.concatenate([GRID, (GRID[1:] + GRID[:-1]) / 2])         # 15 values


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


def _neighbours(v, kind):
    """Float32 values, each with the next one below and above in the type."""
    if kind == "f32":
        return np.concatenate([np.nextafter(v, np.float32(-np.inf)), v, np.nextafter(v, np.float32(np.inf))])
    bits = (v.view(np.uint32) >> 16).astype(np.int64)              # magnitudes, and 0 has no lower one
    low, high = np.maximum(bits - 1, 0), bits + 1
    return np.concatenate([(b.astype(np.uint32) << 16).view(np.float32) for b in (low, bits, high)])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_quantiser_over_every_scale(moe, kind):
    """Scale bytes 0 to 252, the largest that a finite value gives; both signs; the largest
    value of a block at either end of its binade and inside."""
    rows = []
    for byte in range(253):
        p = byte - 127
        v = _neighbours(np.ldexp(POINTS, p).astype(np.float32), kind)
        v = np.concatenate([v, -v])
        top = np.ldexp([1.0, 1.25, 1.9921875], p + 2).astype(np.float32)        # 4, 5 and 7.97 times 2^p
        if byte == 0:
            top = np.append(top, np.ldexp([1.0, 0.25, 3.5], p).astype(np.float32))      # as every smaller one
        for t in top:
            below = v[np.abs(v) <= t]
            below = np.concatenate([below, np.zeros(-len(below) % 31, np.float32)])
            for part in below.reshape(-1, 31):
                rows.append(np.append(part, t))
    x = np.stack(rows).astype(np.float32)
    assert np.isfinite(x).all()
    if kind == "bf16":
        assert np.array_equal(x, (x.view(np.uint32) & 0xFFFF0000).view(np.float32))
    t, v = _tensor(x, kind)
    assert np.array_equal(v, x.astype(np.float64))
    code, byte = mx.quant(v)
    assert len(np.unique(byte)) == 253
    want_q, want_e, want_v = _want(v)
    log(f"mxfp4_quant_1x32 over every scale, {len(x)} blocks {kind}")
    q, e, values = moe.mxfp4_quant_1x32(t, values=True)
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(e.cpu().numpy(), want_e)
    assert _same_values(values, want_v)
    log(f"mxfp4_quant_32x1 over every scale {kind}")
    q, e = moe.mxfp4_quant_32x1(t.t().contiguous())
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(e.cpu().numpy(), want_e)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_reader_over_every_scale_and_code(moe, kind):
    """Every byte, 255 among them, with every code; 6 and 4 at the top two pass the types' range."""
    byte = np.arange(256, dtype=np.uint8)[:, None]
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    q, e = mx.pack(code, byte)
    want = mx.values(code, byte, 32)
    want[np.abs(want) >= 2.0 ** 128] *= np.inf
    log(f"mxfp4_dequant_1x32 over every scale and code {kind}")
    out = moe.mxfp4_dequant_1x32(to_dev(q), to_dev(e), 32,
                                 out_dtype={"bf16": torch.bfloat16, "f32": torch.float32}[kind])
    assert _same_values(out, want)
    got = synth.as_f64(out.view(torch.int16).cpu().numpy().view(np.uint16)) if kind == "bf16" \
        else out.double().cpu().numpy()
    assert np.array_equal(np.signbit(got[:255]), np.signbit(want[:255]))


@pytest.mark.parametrize("rows", [254, 20])
def test_product_over_every_pair_of_scales(moe, rows):
    """Each scale of A with each of B, in row tiles and (few rows) with the weights streamed: a sum
    over one block is a multiple of 1/4 below 2^12 times the scales' product, exact in
    float wherever it is neither subnormal nor too large."""
    rng = np.random.default_rng(rows)
    K = 32
    a_byte = (np.arange(254) if rows == 254 else np.linspace(0, 254, rows).astype(int)).astype(np.uint8)[:, None]
    b_byte = np.arange(255, dtype=np.uint8)[:, None]
    a_code, b_code = (rng.integers(0, 16, (len(b), K), dtype=np.uint8) for b in (a_byte, b_byte))
    (a_q, a_e), (b_q, b_e) = mx.pack(a_code, a_byte), mx.pack(b_code, b_byte)
    want = mx.values(a_code, a_byte) @ mx.values(b_code, b_byte).T
    off = to_dev(np.array([0, rows], np.int32))
    log(f"moe_grouped_gemm_mxfp4 over every pair of scales, {rows} rows")
    out, _ = moe.moe_grouped_gemm_mxfp4(to_dev(a_q), to_dev(a_e), to_dev(b_q)[None], to_dev(b_e)[None], off, rows,
                                        out_dtype=torch.float32, k_dim=K)
    out = out.double().cpu().numpy()
    size = np.abs(want)
    normal = (size >= 2.0 ** -126) & (size < 2.0 ** 128) | (want == 0)
    # the sum of magnitudes stays in range, too
    mag = np.abs(mx.values(a_code, a_byte)) @ np.abs(mx.values(b_code, b_byte)).T
    exact = normal & (mag < 2.0 ** 128)
    assert exact.sum() > want.size // 2
    assert np.array_equal(out[exact], want[exact])
    small = size < 2.0 ** -126                    # a subnormal result may have been flushed to zero
    assert np.all(np.abs(out[small]) < 2.0 ** -126)
    assert not np.isnan(out[mag < 2.0 ** 128]).any()
