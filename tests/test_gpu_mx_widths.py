"""The quantiser and the reader of the 4-bit format at the widths and counts where their
indexes end: rows of almost 2^31 columns, and as many pieces of rows as one dimension of a
launch holds.  Everything is compared bit for bit with the same values cut into short rows,
and those with the float64 oracle."""
import numpy as np
import pytest

from helpers import log
from test_gpu_mx import _hard, _same_values, _tensor, _want

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("cols", [2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 520])
def test_one_row_of_almost_2_31_columns(moe, cols):
    """The last widths a row may have; the sum of columns and a block passes 2^31."""
    period, piece = 1024, 512
    v = _hard(np.random.default_rng(cols % 1000), period, piece)
    part, pv = _tensor(v, "bf16")
    whole = cols // (period * piece)
    rest = cols - whole * period * piece
    x = part.view(-1).repeat(whole + 1)[:cols].view(1, cols)
    log(f"mxfp4_quant_1x32 1 x {cols}")
    q, e, values = moe.mxfp4_quant_1x32(x, values=True)
    want_q, want_e, want_v = moe.mxfp4_quant_1x32(part, values=True)
    oracle_q, oracle_e, oracle_v = _want(pv)
    assert np.array_equal(want_q.cpu().numpy(), oracle_q) and np.array_equal(want_e.cpu().numpy(), oracle_e)
    assert _same_values(want_v, oracle_v)
    tail_q, tail_e, tail_v = moe.mxfp4_quant_1x32(x[:, cols - rest:].clone(), values=True)
    bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t      # noqa: E731  (NaN too)

    def same(got, want, tail):
        got, want, tail = bits(got).view(-1), bits(want).view(-1), bits(tail).view(-1)
        n = whole * want.numel()
        return (got[:n].view(whole, -1) == want).all() and torch.equal(got[n:], tail)
    assert same(q, want_q, tail_q)
    assert same(e, want_e, tail_e)
    assert same(values, want_v, tail_v)
    del values
    log(f"mxfp4_dequant_1x32 1 x {cols}")
    assert same(moe.mxfp4_dequant_1x32(q, e, cols), want_v, tail_v)


@pytest.mark.parametrize("rows", [2 ** 24 - 1, 2 ** 24, 2 ** 24 + 5])
def test_as_many_pieces_as_one_dimension_of_a_launch_holds(moe, rows):
    """2^24 pieces of a row: more go on along the launch's second dimension."""
    period, cols = 1024, 3
    part, pv = _tensor(_hard(np.random.default_rng(rows % 100), period, cols), "f32")
    x = part.repeat(-(-rows // period), 1)[:rows]
    log(f"mxfp4_quant_1x32 {rows} x {cols}")
    q, e, values = moe.mxfp4_quant_1x32(x, values=True)
    want_q, want_e, want_v = _want(pv)
    times = lambda w: torch.from_numpy(w).cuda().repeat(-(-rows // period), 1)[:rows]     # noqa: E731
    assert torch.equal(q, times(want_q)) and torch.equal(e, times(want_e))
    log(f"mxfp4_dequant_1x32 {rows} x {cols}")
    back = moe.mxfp4_dequant_1x32(q, e, cols)
    want = times(want_v)
    for got in (values, back):
        assert torch.equal(got.double().nan_to_num(7e300), want.nan_to_num(7e300))
