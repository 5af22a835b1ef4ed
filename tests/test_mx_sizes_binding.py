"""Sizes of 2^31 and more, which the C entry points take as 32 bit integers, are refused by
the binding and never cut to their low bits.  On the CPU: tensors without storage that
claim to be on the device, and a library that only returns."""
import pytest

torch = pytest.importorskip("torch")

import fp8_block_scaled_sigmoid_amd as moe  # noqa: E402
from test_binding_streams import Device, Library  # noqa: E402

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
MANY = 2 ** 32 + 5                  # 5 in the low bits


def big(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(Device)


CALLS = {
    "quant rows": lambda n: moe.mxfp4_quant_1x32(big(n, 1)),
    "quant batch": lambda n: moe.mxfp4_quant_1x32(big(n, 1, 1)),
    "quant columns": lambda n: moe.mxfp4_quant_1x32(big(1, n)),
    "turned rows": lambda n: moe.mxfp4_quant_32x1(big(n, 1)),
    "turned columns": lambda n: moe.mxfp4_quant_32x1(big(1, n)),
    "reader rows": lambda n: moe.mxfp4_dequant_1x32(big(n, 16, dtype=U8), big(n, 16, dtype=U8), 1),
    "reader columns": lambda n: moe.mxfp4_dequant_1x32(
        big(1, moe.mxfp4_code_bytes(n), dtype=U8), big(1, moe.mxfp4_scale_bytes(n), dtype=U8), n),
    "product rows": lambda n: moe.moe_grouped_gemm_mxfp4(
        big(n, 16, dtype=U8), big(n, 16, dtype=U8), big(1, 1, 16, dtype=U8), big(1, 1, 16, dtype=U8),
        big(2, dtype=I32), n),
    "product gathered": lambda n: moe.moe_grouped_gemm_mxfp4(
        big(n, 16, dtype=U8), big(n, 16, dtype=U8), big(1, 1, 16, dtype=U8), big(1, 1, 16, dtype=U8),
        big(2, dtype=I32), 3, a_row_index=big(3, dtype=I32)),
    "product columns": lambda n: moe.moe_grouped_gemm_mxfp4(
        big(3, 16, dtype=U8), big(3, 16, dtype=U8), big(1, n, 16, dtype=U8), big(1, n, 16, dtype=U8),
        big(2, dtype=I32), 3),
    "loss tokens": lambda n: moe.moe_balance_loss(big(n, 1, dtype=F32), big(n, 1, dtype=I32)),
    "loss experts": lambda n: moe.moe_balance_loss(big(1, n, dtype=F32), big(1, 1, dtype=I32)),
    "loss picks": lambda n: moe.moe_balance_loss(big(1, 8, dtype=F32), big(1, n, dtype=I32)),
    "loss sequences": lambda n: moe.moe_balance_loss(big(3, 1, dtype=F32), big(3, 1, dtype=I32),
                                                     big(n + 1, dtype=I32)),
    "gradient tokens": lambda n: moe.moe_router_backward(big(n, 1, dtype=F32), big(n, 1, dtype=I32)),
    "gradient sequences": lambda n: moe.moe_router_backward(big(3, 1, dtype=F32), big(3, 1, dtype=I32),
                                                            seq_offsets=big(n + 1, dtype=I32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused(monkeypatch, name):
    monkeypatch.setattr(moe, "lib", lambda: Library())
    monkeypatch.setattr(moe, "_queue", lambda stream: 0)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **{**k, "device": "meta"}).as_subclass(Device))
    assert CALLS[name](5) is not None               # the same call with a small size goes through
    for n in (2 ** 31, MANY):
        with pytest.raises(ValueError, match="2\\^31"):
            CALLS[name](n)
