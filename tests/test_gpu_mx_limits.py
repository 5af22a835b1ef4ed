"""The 4-bit product at the ends of its documented ranges: operands of almost 2^31 bytes,
rows far apart, a very long k, and a gated result with strided rows.  All scales are 1 and
every sum is a multiple of 1/4 below 2^22, so that a float result is exact."""
import numpy as np
import pytest

from helpers import log, to_dev
from oracle import mx
from test_gpu_mx import _offsets, _operand

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("R", [130, 20])
def test_the_most_columns(moe, R):
    """126,322,000 rows of B, 2.02 GB of codes and as many of scales, of one pattern."""
    n, K, period = 126_322_000, 5, 50_000
    rng = np.random.default_rng(R)
    a_q, a_e, a = _operand(rng, R, K, 0)
    p_q, p_e, p = _operand(rng, period, K, 0)
    times = -(-n // period)
    b_q, b_e = p_q.repeat(times, 1)[None, :n], p_e.repeat(times, 1)[None, :n]
    log(f"moe_grouped_gemm_mxfp4 {R} x {n}")
    out, _ = moe.moe_grouped_gemm_mxfp4(a_q, a_e, b_q, b_e, to_dev(np.array([0, R], np.int32)), R, k_dim=K)
    want = to_dev(np.ascontiguousarray((a @ p.T).astype(np.float32))).bfloat16()
    for r in range(R):
        whole = n // period * period
        assert (out[r, :whole].view(-1, period) == want[r]).all(), r
        assert torch.equal(out[r, whole:], want[r, :n - whole]), r


@pytest.mark.parametrize("sizes,K", [([288], 11_000_064), ([150, 129], 11_000_001), ([33], 11_000_001)], ids=str)
def test_the_longest_rows(moe, sizes, K):
    """k of 11 million, codes of 0 and +-1/2: 1.6 GB of A, 1.07 GB of B a group."""
    n, off, R, G = 194, _offsets(sizes), sum(sizes), len(sizes)
    gen = torch.Generator(device="cuda").manual_seed(R)
    cb, sb = moe.mxfp4_code_bytes(K), moe.mxfp4_scale_bytes(K)
    table = torch.tensor([0, 1, 9], dtype=torch.uint8, device="cuda")

    def operand(*lead):
        low, high = (table[torch.randint(0, 3, (*lead, cb), device="cuda", generator=gen)] for _ in range(2))
        q = low | high << 4
        if K % 32:                      # the missing columns of the last block
            q[..., K // 2] &= 15
            q[..., (K + 1) // 2:] = 0
        return q, torch.full((*lead, sb), 127, dtype=torch.uint8, device="cuda")
    a_q, a_e = operand(R)
    b_q, b_e = operand(G, n)
    log(f"moe_grouped_gemm_mxfp4 {sizes} x {n} x {K}")
    out, _ = moe.moe_grouped_gemm_mxfp4(a_q, a_e, b_q, b_e, to_dev(off), R, out_dtype=torch.float32, k_dim=K)
    want = torch.zeros(R, n, dtype=torch.float64, device="cuda")
    part = 1 << 20                      # columns at a time, whole pieces of scales
    for at in range(0, K, part):
        cols = min(part, K - at)
        codes = slice(at // 2, at // 2 + moe.mxfp4_code_bytes(cols))
        scales = slice(at // 32, at // 32 + moe.mxfp4_scale_bytes(cols))
        read = lambda q, e: moe.mxfp4_dequant_1x32(q[..., codes].contiguous(), e[..., scales].contiguous(), cols,  # noqa: E731,E501
                                                   out_dtype=torch.float32)
        rows, weights = read(a_q, a_e), read(b_q, b_e)
        for g in range(G):                      # exact: multiples of 1/4 below 2^19
            lo, hi = int(off[g]), int(off[g + 1])
            want[lo:hi] += (rows[lo:hi] @ weights[g].t()).double()
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("K", [512, 600])
def test_rows_of_A_far_apart(moe, gathered, K):
    """Codes and scales at a stride of 7.4 MB: 288 rows take 2^31 bytes less 3584."""
    R, n, stride = 288, 260, 7_456_528
    rng = np.random.default_rng(K + gathered)
    q, e, a = _operand(rng, R, K, 0)
    b_q, b_e, b = _operand(rng, n, K, 0)
    spread = lambda t: torch.full((R * stride,), 255, dtype=torch.uint8, device="cuda").view(  # noqa: E731
        R, stride)[:, :t.shape[1]].copy_(t)
    a_q, a_e = spread(q), spread(e)
    assert a_q.stride(0) == stride and a_e.stride(0) == stride
    order = np.arange(R)[::-1].astype(np.int32).copy() if gathered else np.arange(R)
    log(f"moe_grouped_gemm_mxfp4 of rows far apart, K={K} gathered={gathered}")
    out, _ = moe.moe_grouped_gemm_mxfp4(a_q, a_e, b_q[None], b_e[None], to_dev(np.array([0, R], np.int32)), R,
                                        a_row_index=to_dev(order) if gathered else None, out_dtype=torch.float32,
                                        k_dim=K)
    assert np.array_equal(out.cpu().numpy(), (a[order] @ b.T).astype(np.float32))


@pytest.mark.parametrize("rows", [[40, 3], [290, 31]], ids=str)
def test_gated_result_in_strided_rows(moe, rows):
    """Codes into rows wider than they are; rows behind the last group are left as they were."""
    I, K = 640, 160
    rng = np.random.default_rng(sum(rows))
    R, G = sum(rows) + 7, len(rows)
    off = to_dev(_offsets(rows))                            # seven rows belong to no group
    a_q, a_e, _ = _operand(rng, R, K, 1)
    b_q, b_e, _ = _operand(rng, G * 2 * I, K, 1)
    b_q, b_e = b_q.view(G, 2 * I, -1), (b_e - 8).view(G, 2 * I, -1)
    run = lambda **kw: moe.moe_grouped_gemm_mxfp4(a_q, a_e, b_q, b_e, off, R, moe.MOE_EPI_SWIGLU_MXFP4,   # noqa: E731
                                                  k_dim=K, **kw)
    width, scales = moe.mxfp4_code_bytes(I), moe.mxfp4_scale_bytes(I)
    buf = torch.full((R + 2, width + 20), 0xA5, dtype=torch.uint8, device="cuda")
    e = torch.full((R + 2, scales), 0xA5, dtype=torch.uint8, device="cuda")
    log(f"moe_grouped_gemm_mxfp4 gated into strided rows {rows}")
    run(out=buf[1:R + 1, 4:width + 4], out_e=e[1:R + 1])
    q, want_e = run()
    n = sum(rows)
    assert torch.equal(buf[1:n + 1, 4:width + 4], q[:n]) and torch.equal(e[1:n + 1], want_e[:n])
    for t in (buf[0], buf[n + 1:], buf[:, :4], buf[:, width + 4:], e[0], e[n + 1:]):
        assert (t == 0xA5).all()
    code, byte = mx.unpack(q[:n].cpu().numpy(), want_e[:n].cpu().numpy())
    assert np.isfinite(mx.values(code, byte)).all() and (code != 0).any()
