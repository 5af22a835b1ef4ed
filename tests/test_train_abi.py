"""The training entry points' C ABI on the CPU: declared, exported, and
rejecting invalid arguments before touching a device."""
import ctypes
import os

import pytest

import fp8_block_scaled_sigmoid_amd as moe
from test_abi import declared_functions

P16 = 16        # a non-NULL, 16-byte aligned pointer that is never followed


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.fail("libmoe_fp8.so is not built (run __graft_entry__.build())")
    return moe.lib()


def test_declared_and_exported(lib):
    names = declared_functions()
    for n in ("moe_block_norm", "moe_block_norm_backward",
              "moe_block_norm_backward_workspace_bytes", "moe_grouped_gemm_bf16",
              "moe_grouped_gemm_bf16_workspace_bytes",
              "moe_grouped_wgrad_bf16", "moe_grouped_wgrad_bf16_workspace_bytes", "moe_swiglu",
              "moe_swiglu_backward", "moe_grad_table_bytes", "moe_grad_table",
              "moe_grad_norm_workspace_bytes", "moe_grad_norm", "moe_grad_scale", "moe_grad_clip"):
        assert n in names and hasattr(lib, n), n


def _args(cls, base, **kw):
    a = cls()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return ctypes.byref(a)


NORM = dict(T=4, H=16, x=P16, ldx=16, b=P16, ldb=16, w_pre=P16, w_post=P16, alpha=1, beta=1,
            eps=1e-6, r=P16, ldr=16, h=P16, ldh=16)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 2), (dict(H=0), 2), (dict(H=16385, ldx=16385), 2), (dict(eps=0.0), 2),
    (dict(eps=float("nan")), 2), (dict(ldx=15), 2), (dict(ldb=15), 2), (dict(ldr=8), 2),
    (dict(ldh=0), 2), (dict(x_dtype=2), 6), (dict(b_dtype=-1), 6), (dict(gate_mode=4), 6),
    (dict(gate_mode=3, gate=P16, ldg=4), 2), (dict(gate_mode=1), 1), (dict(x=None), 1),
    (dict(r=None), 1), (dict(w_pre=None), 1), (dict(b=None, h=None), 1), (dict(x=17), 3),
    (dict(x_dtype=1, x=18), 3), (dict(w_pre=18), 3), (dict(T=0, x=None), 0)])
def test_block_norm_arguments(lib, change, status):
    assert lib.moe_block_norm(_args(moe.BlockNormArgs, NORM, **change), None) == status


BWD = dict(T=4, H=16, r=P16, ldr=16, dr=P16, lddr=16, dh=P16, lddh=16, b=P16, ldb=16, w_pre=P16,
           w_post=P16, alpha=1, beta=1, eps=1e-6, dx=P16, lddx=16, db=P16, lddb=16, dw_pre=P16,
           dw_post=P16)


@pytest.mark.parametrize("change,status", [
    (dict(H=20000), 2), (dict(eps=-1.0), 2), (dict(lddx=8), 2), (dict(dr=None, dh=None), 1),
    (dict(r=None), 1), (dict(dh=None), 1), (dict(b=None), 1), (dict(w_post=None), 1),
    (dict(dgate=P16), 1), (dict(gate_mode=2), 1), (dict(db=17), 3), (dict(), 4),
    (dict(T=0, dw_pre=None, dw_post=None), 0)])
def test_block_norm_backward_arguments(lib, change, status):
    assert lib.moe_block_norm_backward(_args(moe.BlockNormBwdArgs, BWD, **change), None, 0,
                                       None) == status


GEMM = dict(a=P16, lda=16, a_rows=4, b=P16, group_offsets=P16, num_groups=2, total_rows=4, n_out=8,
            k_dim=16, out=P16, ldo=8)


@pytest.mark.parametrize("change,status", [
    (dict(n_out=12, ldo=16), 2), (dict(k_dim=12), 2), (dict(lda=8), 2), (dict(lda=20), 2),
    (dict(ldo=4), 2), (dict(a_rows=3), 2), (dict(num_groups=0), 2), (dict(num_groups=1026), 6),
    (dict(out_dtype=2), 6), (dict(b_layout=2), 6),
    (dict(a_row_index=P16, a_rows=1 << 28), 6),
    (dict(n_out=1 << 20, ldo=1 << 20, k_dim=1 << 10, lda=1 << 10), 6), (dict(a=None), 1),
    (dict(group_offsets=None), 1), (dict(out=None), 1), (dict(b=24), 3), (dict(total_rows=0), 0),
    (dict(n_out=0), 0)])
def test_grouped_gemm_arguments(lib, change, status):
    assert lib.moe_grouped_gemm_bf16(_args(moe.GemmBf16Args, GEMM, **change), None, 0, None) == status


def test_block_norm_refuses_more_rows_than_its_counters_hold(lib):
    assert lib.moe_block_norm(_args(moe.BlockNormArgs, NORM, T=(1 << 30) + 1), None) == 6
    assert lib.moe_block_norm_backward(_args(moe.BlockNormBwdArgs, BWD, T=(1 << 30) + 1), None, 0,
                                       None) == 6


@pytest.mark.parametrize("change,status", [
    (dict(b_layout=1, n_out=1 << 24, ldo=1 << 24), 6),      # a step's rows of B pass 32 bits
    (dict(lda=1 << 22), 6), (dict(n_out=1 << 26, ldo=1 << 26, total_rows=0), 6)])
def test_grouped_gemm_refuses_sizes_past_its_offsets(lib, change, status):
    assert lib.moe_grouped_gemm_bf16(_args(moe.GemmBf16Args, GEMM, **change), None, 0, None) == status


def test_grouped_gemm_workspace(lib):
    need = lib.moe_grouped_gemm_bf16_workspace_bytes
    assert need(33, 144, 4096, 7168) == 0           # few rows a group: the weights' stream
    assert need(1, 1000, 1024, 512) == 0            # a tile for every workgroup at most
    assert need(33, 16384, 4096, 7168) > 0
    assert need(0, 16384, 4096, 7168) == 0 and need(33, 0, 4096, 7168) == 0
    many = dict(a_rows=1 << 17, total_rows=1 << 17, n_out=1024, ldo=1024)
    assert lib.moe_grouped_gemm_bf16(_args(moe.GemmBf16Args, GEMM, **many), None, 0, None) == 4
    assert lib.moe_grouped_gemm_bf16(_args(moe.GemmBf16Args, GEMM, **many), 24, 512, None) == 3


WGRAD = dict(a=P16, lda=8, a_rows=4, b=P16, ldb=16, b_rows=4, group_offsets=P16, num_groups=2,
             total_rows=4, n=8, k=16, out=P16)


@pytest.mark.parametrize("change,status", [
    (dict(n=12, lda=16), 2), (dict(k=20, ldb=24), 2), (dict(lda=4), 2), (dict(ldb=12), 2),
    (dict(a_rows=3), 2), (dict(b_rows=3), 2), (dict(num_groups=0), 2), (dict(num_groups=1026), 6),
    (dict(b_row_index=P16, b_rows=1 << 28), 6), (dict(out_dtype=3), 6), (dict(b=None), 1),
    (dict(out=None), 1), (dict(out=8), 3), (dict(n=0), 0)])
def test_grouped_wgrad_arguments(lib, change, status):
    assert lib.moe_grouped_wgrad_bf16(_args(moe.WgradBf16Args, WGRAD, **change), None, 0,
                                      None) == status


def test_grouped_wgrad_workspace(lib):
    need = lib.moe_grouped_wgrad_bf16_workspace_bytes
    assert need(33, 16384, 4096, 7168) == 0             # tiles enough for every compute unit
    assert need(1, 8192, 256, 7168) > 0 and need(1, 100, 256, 7168) == 0
    assert need(0, 8192, 256, 256) == 0 and need(1, 8192, 0, 256) == 0
    long = dict(a_rows=8192, b_rows=8192, total_rows=8192, num_groups=1)
    assert lib.moe_grouped_wgrad_bf16(_args(moe.WgradBf16Args, WGRAD, **long), None, 0, None) == 4
    assert lib.moe_grouped_wgrad_bf16(_args(moe.WgradBf16Args, WGRAD, **long), 24, 1 << 30, None) == 3


def test_swiglu_arguments(lib):
    f = lambda a=P16, dt=0, R=4, I=8, lda=16, h=P16, ldh=8: lib.moe_swiglu(  # noqa: E731
        a, dt, R, I, lda, h, ldh, None)
    assert f(R=-1) == 2 and f(lda=15) == 2 and f(ldh=7) == 2 and f(dt=2) == 6
    assert f(a=None) == 1 and f(a=17) == 3 and f(R=0, a=None) == 0 and f(I=0) == 0
    b = lambda dh=P16, lddh=8, ldda=16, hg=None, ldhg=8, da=P16: lib.moe_swiglu_backward(  # noqa: E731
        P16, dh, 1, 4, 8, 16, lddh, None, da, ldda, None, hg, ldhg, None)
    assert b(lddh=4) == 2 and b(ldda=8) == 2 and b(hg=P16, ldhg=4) == 2
    assert b(dh=None) == 1 and b(da=18) == 3


def test_grad_table_and_calls(lib):
    def table(*rows, room=1000):
        buf, chunks = ctypes.create_string_buffer(1000), ctypes.c_longlong(-1)
        arr = (moe.GradTensor * max(len(rows), 1))(*[moe.GradTensor(*r) for r in rows])
        return lib.moe_grad_table(arr, len(rows), buf, room, ctypes.byref(chunks)), chunks.value
    assert lib.moe_grad_table_bytes(3) == 120 and lib.moe_grad_table_bytes(0) == 0
    status, chunks = table((4096, 4096, 16385, 1, 1), (0, 0, 0, 1, 1), (1 << 20, 1 << 20, 5, 0, 0))
    assert status == 0 and chunks >= 2           # one at least for every tensor with elements
    assert table()[0] == 0
    assert table((4096, 4096, 10, 1, 1), room=39)[0] == 4
    assert table((4096, 4096, -1, 1, 1))[0] == 2
    assert table((4096, 4096, 10, 2, 1))[0] == 6
    assert table((None, 4096, 10, 1, 1))[0] == 1
    assert table((4098, 8192, 10, 1, 1))[0] == 3
    assert table((4096, 4096, 10, 1, 0))[0] == 6                            # in place, two types
    assert table((4096, 4100, 10, 1, 1))[0] == 6                            # partly its own source
    assert table((4096, 8192, 10, 1, 1), (8200, 16384, 10, 1, 1))[0] == 6     # another's source
    assert table((4096, 8192, 10, 1, 1), (16384, 8228, 10, 1, 1))[0] == 6     # another's destination
    assert table((4096, 8192, 10, 1, 1), (4096, 16384, 10, 1, 1))[0] == 0     # read twice
    assert lib.moe_grad_norm_workspace_bytes(0) == 8
    assert lib.moe_grad_norm_workspace_bytes(10 ** 9) == 2048 * 8
    assert lib.moe_grad_clip(P16, 1, -1, P16, 8, 1.0, None, None) == 2
    assert lib.moe_grad_clip(P16, 1, 1, P16, 8, -1.0, None, None) == 2
    assert lib.moe_grad_clip(P16, 1, 1, P16, 8, float("nan"), None, None) == 2
    assert lib.moe_grad_clip(P16, 1, 1, None, 8, 1.0, None, None) == 4
    assert lib.moe_grad_clip(P16, 1, 4, P16, 8, 1.0, None, None) == 4
    assert lib.moe_grad_clip(None, 1, 1, P16, 8, 1.0, None, None) == 1
    assert lib.moe_grad_clip(20, 1, 1, P16, 8, 1.0, None, None) == 3
    assert lib.moe_grad_norm(P16, 1, 1, P16, 8, None, None, None) == 1
    assert lib.moe_grad_scale(P16, 1, 1, None, 1.0, None, None) == 1
