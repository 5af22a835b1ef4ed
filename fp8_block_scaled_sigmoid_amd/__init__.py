"""Python binding of libmoe_fp8.so: the DeepSeekMoE forward layer on MI355X.

Argument marshalling only.  Every step of the layer runs in the HIP kernels
behind the C ABI declared in ``include/moe_fp8.h``; PyTorch is used for device
memory and the current stream, nothing else.  There is no fallback: if the
library is missing or the device is not gfx950 the calls raise.

The functions carry the C entry points' names.  ``MoELayer`` chains them into
the forward pass (router + biased top-k, permutation, 1x128 activation
quantisation, the two grouped FP8 GEMMs, combine, bias update);
``moe_layer_forward`` runs the same steps in one library call.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_fp8.so")

MOE_BF16, MOE_F32 = 0, 1
MOE_EPI_BF16, MOE_EPI_SWIGLU_FP8, MOE_EPI_F32, MOE_EPI_SWIGLU_MXFP4 = 0, 1, 2, 3
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_FULL = 0, 1, 2, 3
MOE_B_NK, MOE_B_KN = 0, 1

STATUS = {0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_ALIGN",
          4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_DEVICE", 6: "MOE_ERR_UNSUPPORTED",
          7: "MOE_ERR_HIP"}


class MoeError(RuntimeError):
    def __init__(self, fn, code, hip=0):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}"
                         + (f" (hipError {hip})" if code == 7 else ""))
        self.code = code


class GemmArgs(ctypes.Structure):
    _fields_ = [("a_q", ctypes.c_void_p), ("a_d", ctypes.c_void_p), ("lda", ctypes.c_int),
                ("a_rows", ctypes.c_int), ("a_row_index", ctypes.c_void_p),
                ("b_q", ctypes.c_void_p), ("b_d", ctypes.c_void_p),
                ("group_offsets", ctypes.c_void_p), ("num_groups", ctypes.c_int),
                ("total_rows", ctypes.c_int), ("n_out", ctypes.c_int), ("k_dim", ctypes.c_int),
                ("epilogue", ctypes.c_int), ("out", ctypes.c_void_p), ("out_d", ctypes.c_void_p),
                ("ldo", ctypes.c_int), ("row_scale", ctypes.c_void_p)]


class LayerArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("w_router", ctypes.c_void_p),
                ("w_router_q", ctypes.c_void_p), ("w_router_d", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("w1_q", ctypes.c_void_p), ("w1_d", ctypes.c_void_p),
                ("w2_q", ctypes.c_void_p), ("w2_d", ctypes.c_void_p),
                ("T", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int), ("k", ctypes.c_int),
                ("I", ctypes.c_int), ("with_shared", ctypes.c_int), ("n_groups", ctypes.c_int),
                ("topk_groups", ctypes.c_int), ("router_fp8", ctypes.c_int),
                ("update_bias", ctypes.c_int), ("gamma", ctypes.c_float),
                ("residual", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("scores", ctypes.c_void_p), ("topk_idx", ctypes.c_void_p),
                ("topk_gate", ctypes.c_void_p), ("counts", ctypes.c_void_p)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_LL = ctypes.c_longlong
_F = ctypes.c_float
_SZ = ctypes.c_size_t


class BlockNormArgs(ctypes.Structure):
    _fields_ = [("T", _I), ("H", _I), ("x_dtype", _I), ("b_dtype", _I),
                ("x", _P), ("ldx", _LL), ("b", _P), ("ldb", _LL), ("w_pre", _P), ("w_post", _P),
                ("gate_mode", _I), ("gate", _P), ("ldg", _LL),
                ("alpha", _F), ("beta", _F), ("eps", _F),
                ("r", _P), ("ldr", _LL), ("h", _P), ("ldh", _LL)]


class BlockNormBwdArgs(ctypes.Structure):
    _fields_ = [("T", _I), ("H", _I), ("x_dtype", _I), ("b_dtype", _I),
                ("r", _P), ("ldr", _LL), ("dr", _P), ("lddr", _LL), ("dh", _P), ("lddh", _LL),
                ("b", _P), ("ldb", _LL), ("w_pre", _P), ("w_post", _P),
                ("gate_mode", _I), ("gate", _P), ("ldg", _LL),
                ("alpha", _F), ("beta", _F), ("eps", _F),
                ("dx", _P), ("lddx", _LL), ("db", _P), ("lddb", _LL),
                ("dw_pre", _P), ("dw_post", _P), ("dgate", _P), ("lddg", _LL)]


class GemmBf16Args(ctypes.Structure):
    _fields_ = [("a", _P), ("lda", _LL), ("a_rows", _I), ("a_row_index", _P), ("b", _P),
                ("b_layout", _I), ("group_offsets", _P), ("num_groups", _I), ("total_rows", _I),
                ("n_out", _I), ("k_dim", _I), ("out_dtype", _I), ("out", _P), ("ldo", _LL),
                ("row_scale", _P)]


class WgradBf16Args(ctypes.Structure):
    _fields_ = [("a", _P), ("lda", _LL), ("a_rows", _I), ("a_row_index", _P),
                ("b", _P), ("ldb", _LL), ("b_rows", _I), ("b_row_index", _P),
                ("group_offsets", _P), ("num_groups", _I), ("total_rows", _I), ("n", _I),
                ("k", _I), ("out_dtype", _I), ("out", _P), ("accumulate", _I)]


class GemmMxfp4Args(ctypes.Structure):
    _fields_ = [("a_q", _P), ("lda", _LL), ("a_e", _P), ("lde", _LL), ("a_rows", _I),
                ("a_row_index", _P), ("b_q", _P), ("b_e", _P), ("group_offsets", _P),
                ("num_groups", _I), ("total_rows", _I), ("n_out", _I), ("k_dim", _I),
                ("epilogue", _I), ("out", _P), ("ldo", _LL), ("out_e", _P), ("row_scale", _P)]


class BalanceArgs(ctypes.Structure):
    _fields_ = [("T", _I), ("N", _I), ("k", _I), ("n_seq", _I), ("scores", _P), ("lds", _LL),
                ("topk_idx", _P), ("seq_offsets", _P), ("token_mask", _P), ("alpha", _F),
                ("loss", _P), ("load", _P), ("prob", _P), ("counts", _P), ("tokens", _P)]


class RouterBwdArgs(ctypes.Structure):
    _fields_ = [("T", _I), ("N", _I), ("k", _I), ("n_seq", _I), ("scores", _P), ("lds", _LL),
                ("topk_idx", _P), ("topk_gate", _P), ("dgate", _P), ("load", _P), ("tokens", _P),
                ("seq_offsets", _P), ("token_mask", _P), ("dloss", _P), ("alpha", _F),
                ("out_dtype", _I), ("dz", _P), ("ldz", _LL)]


class GradTensor(ctypes.Structure):
    _fields_ = [("src", _P), ("dst", _P), ("numel", _LL), ("src_dtype", _I), ("dst_dtype", _I)]


def lib():
    """Load libmoe_fp8.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "moe_route_topk": [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, ctypes.c_size_t, _P],
            "moe_route_topk_quant_x": [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P,
                                       ctypes.c_size_t, _P],
            "moe_route_topk_fp8": [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                   ctypes.c_size_t, _P],
            "moe_topk_from_scores": [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P],
            "moe_permute": [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
            "fp8_quant_1x128": [_P, _I, _I, _I, _I, _P, _P, _P],
            "fp8_quant_128x128": [_P, _I, _I, _I, _I, _P, _P, _P],
            "moe_grouped_gemm_fp8": [ctypes.POINTER(GemmArgs), _P],
            "moe_grouped_gemm_fp8_tiles": [ctypes.POINTER(GemmArgs), _I, _P],
            "moe_combine": [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P],
            "moe_bias_update": [_P, _P, _I, _I, _I, ctypes.c_float, _P],
            "moe_seq_balance_loss": [_P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P, _P],
            "fp8_transpose_128x128": [_P, _P, _I, _I, _I, _P, _P, _P],
            "fp8_quant_tokens_128": [_P, _I, _I, _I, _LL, _P, _I, _P, _P, _LL, _P, _P],
            "moe_grouped_wgrad_fp8": [_P, _P, _LL, _I, _P, _P, _LL, _I, _P, _I, _P, _P],
            "moe_probe_fp8_mfma": [_I, _I, _P, _P],
            "moe_probe_hbm": [_I, _P, ctypes.c_size_t, _P, _P],
            "moe_permute_noalloc": [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P],
            "moe_layer_forward": [ctypes.POINTER(LayerArgs), _P, ctypes.c_size_t, _P],
            "moe_block_norm": [ctypes.POINTER(BlockNormArgs), _P],
            "moe_block_norm_backward": [ctypes.POINTER(BlockNormBwdArgs), _P, _SZ, _P],
            "moe_grouped_gemm_bf16": [ctypes.POINTER(GemmBf16Args), _P, _SZ, _P],
            "moe_grouped_wgrad_bf16": [ctypes.POINTER(WgradBf16Args), _P, _SZ, _P],
            "moe_swiglu": [_P, _I, _I, _I, _LL, _P, _LL, _P],
            "moe_swiglu_backward": [_P, _P, _I, _I, _I, _LL, _LL, _P, _P, _LL, _P, _P, _LL, _P],
            "moe_grad_table": [ctypes.POINTER(GradTensor), _I, _P, _SZ, ctypes.POINTER(_LL)],
            "moe_grad_norm": [_P, _I, _LL, _P, _SZ, _P, _P, _P],
            "moe_grad_scale": [_P, _I, _LL, _P, _F, _P, _P],
            "moe_grad_clip": [_P, _I, _LL, _P, _SZ, _F, _P, _P],
            "mxfp4_quant_1x32": [_P, _I, _I, _I, _I, _LL, _I, _P, _P, _P, _P],
            "mxfp4_quant_32x1": [_P, _I, _I, _I, _I, _LL, _P, _P, _P],
            "mxfp4_dequant_1x32": [_P, _P, _I, _I, _I, _P, _LL, _P],
            "moe_grouped_gemm_mxfp4": [ctypes.POINTER(GemmMxfp4Args), _P, _SZ, _P],
            "moe_balance_loss": [ctypes.POINTER(BalanceArgs), _P, _SZ, _P],
            "moe_router_backward": [ctypes.POINTER(RouterBwdArgs), _P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.moe_permute_workspace_bytes.argtypes = [_I, _I, _I]
        L.moe_permute_workspace_bytes.restype = ctypes.c_size_t
        L.moe_route_workspace_bytes.argtypes = [_I, _I, _I]
        L.moe_route_workspace_bytes.restype = ctypes.c_size_t
        L.moe_permute_noalloc_max_scratch_bytes.argtypes = []
        L.moe_permute_noalloc_max_scratch_bytes.restype = ctypes.c_size_t
        L.moe_layer_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
        L.moe_layer_workspace_bytes.restype = ctypes.c_size_t
        L.moe_block_norm_backward_workspace_bytes.argtypes = [_I, _I]
        L.moe_block_norm_backward_workspace_bytes.restype = _SZ
        L.moe_grouped_gemm_bf16_workspace_bytes.argtypes = [_I, _I, _I, _I]
        L.moe_grouped_gemm_bf16_workspace_bytes.restype = _SZ
        L.moe_grouped_wgrad_bf16_workspace_bytes.argtypes = [_I, _I, _I, _I]
        L.moe_grouped_wgrad_bf16_workspace_bytes.restype = _SZ
        L.moe_grad_table_bytes.argtypes = [_I]
        L.moe_grad_table_bytes.restype = _SZ
        L.moe_grad_norm_workspace_bytes.argtypes = [_LL]
        L.moe_grad_norm_workspace_bytes.restype = _SZ
        L.moe_grouped_gemm_mxfp4_workspace_bytes.argtypes = [_I, _I, _I, _I]
        L.moe_grouped_gemm_mxfp4_workspace_bytes.restype = _SZ
        L.moe_balance_loss_workspace_bytes.argtypes = [_I, _I, _I]
        L.moe_balance_loss_workspace_bytes.restype = _SZ
        L.moe_status_str.argtypes = [_I]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_last_hip_error.argtypes = []
        L.moe_last_hip_error.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(name, rc):
    if rc != 0:
        raise MoeError(name, rc, lib().moe_last_hip_error() if rc == 7 else 0)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, dtype, name):
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{name}: need a contiguous {dtype} device tensor, got "
                         f"{t.dtype} on {t.device} (contiguous={t.is_contiguous()})")
    return t


def _allocator(stream, make=None):
    """torch.empty (or `make`) for a call on `stream`: the memory belongs to
    that stream, so that the allocator gives it to later work of that stream
    only, also where the call drops it with its kernels still to run.  The
    caller's stream is noted as well, where the caller will read and drop a
    result."""
    make = make or torch.empty
    if stream is None:
        return make

    def on_stream(*shape, **kw):
        with torch.cuda.stream(stream):
            t = make(*shape, **kw)
        t.record_stream(torch.cuda.current_stream())
        return t
    return on_stream


# ---------------------------------------------------------------------------
# the C entry points


def moe_route_workspace_bytes(T, H, N):
    return int(lib().moe_route_workspace_bytes(T, H, N))


def moe_route_topk(x, w_router, bias, k, scores=True, idx=None, gate=None, ws=None,
                   n_groups=1, topk_groups=1, stream=None):
    """Sigmoid router + biased top-k.  x [T,H] bf16, w_router [N,H] bf16,
    bias [N] float32.  Returns (idx int32 [T,k], gate float32 [T,k],
    scores float32 [T,N] or None).  ws: optional uint8 device scratch of
    moe_route_workspace_bytes(T, H, N) bytes.  n_groups > 1 turns on the
    group-limited selection (the best topk_groups groups are eligible)."""
    empty = _allocator(stream)
    T, H = x.shape
    N = w_router.shape[0]
    _dev(x, torch.bfloat16, "x"), _dev(w_router, torch.bfloat16, "w_router")
    _dev(bias, torch.float32, "bias")
    if scores is True:
        scores = empty(T, N, dtype=torch.float32, device=x.device)
    elif scores is False:
        scores = None
    idx = empty(T, k, dtype=torch.int32, device=x.device) if idx is None else idx
    gate = empty(T, k, dtype=torch.float32, device=x.device) if gate is None else gate
    if ws is None:
        ws = empty(max(moe_route_workspace_bytes(T, H, N), 16), dtype=torch.uint8,
                   device=x.device)
    _check("moe_route_topk", lib().moe_route_topk(_ptr(x), _ptr(w_router), _ptr(bias), T, H, N, k,
                                                  n_groups, topk_groups, _ptr(scores), _ptr(idx),
                                                  _ptr(gate), _ptr(ws), ws.numel(), _stream(stream)))
    return idx, gate, scores


def moe_route_topk_quant_x(x, w_router, bias, k, x_q=None, x_d=None, scores=True, idx=None,
                           gate=None, ws=None, n_groups=1, topk_groups=1, stream=None):
    """moe_route_topk that also writes the 1x128 FP8 quantisation of x (the
    codes and scales fp8_quant_1x128 gives) from the same read of x.
    Returns (idx, gate, scores, x_q uint8 [T,H], x_d float32 [T,H/128])."""
    empty = _allocator(stream)
    T, H = x.shape
    N = w_router.shape[0]
    _dev(x, torch.bfloat16, "x"), _dev(w_router, torch.bfloat16, "w_router")
    _dev(bias, torch.float32, "bias")
    if scores is True:
        scores = empty(T, N, dtype=torch.float32, device=x.device)
    elif scores is False:
        scores = None
    idx = empty(T, k, dtype=torch.int32, device=x.device) if idx is None else idx
    gate = empty(T, k, dtype=torch.float32, device=x.device) if gate is None else gate
    x_q = empty(T, H, dtype=torch.uint8, device=x.device) if x_q is None else x_q
    x_d = empty(T, H // 128, dtype=torch.float32, device=x.device) if x_d is None else x_d
    _dev(x_q, torch.uint8, "x_q"), _dev(x_d, torch.float32, "x_d")
    if ws is None:
        ws = empty(max(moe_route_workspace_bytes(T, H, N), 16), dtype=torch.uint8,
                   device=x.device)
    _check("moe_route_topk_quant_x",
           lib().moe_route_topk_quant_x(_ptr(x), _ptr(w_router), _ptr(bias), T, H, N, k, n_groups,
                                        topk_groups, _ptr(scores), _ptr(idx), _ptr(gate),
                                        _ptr(x_q), _ptr(x_d), _ptr(ws), ws.numel(),
                                        _stream(stream)))
    return idx, gate, scores, x_q, x_d


def moe_route_topk_fp8(x_q, x_d, w_router_q, w_router_d, bias, k, scores=True, idx=None,
                       gate=None, ws=None, n_groups=1, topk_groups=1, stream=None):
    """Opt-in FP8 router + biased top-k.  x_q uint8 [T,H] with x_d float32
    [T,H/128] (fp8_quant_1x128), w_router_q uint8 [N,H] with w_router_d float32
    [N/128,H/128] (fp8_quant_128x128), bias [N] float32.  Same outputs and
    workspace as moe_route_topk."""
    empty = _allocator(stream)
    T, H = x_q.shape
    N = w_router_q.shape[-2]
    _dev(x_q, torch.uint8, "x_q"), _dev(x_d, torch.float32, "x_d")
    _dev(w_router_q, torch.uint8, "w_router_q"), _dev(w_router_d, torch.float32, "w_router_d")
    _dev(bias, torch.float32, "bias")
    if scores is True:
        scores = empty(T, N, dtype=torch.float32, device=x_q.device)
    elif scores is False:
        scores = None
    idx = empty(T, k, dtype=torch.int32, device=x_q.device) if idx is None else idx
    gate = empty(T, k, dtype=torch.float32, device=x_q.device) if gate is None else gate
    if ws is None:
        ws = empty(max(moe_route_workspace_bytes(T, H, N), 16), dtype=torch.uint8,
                   device=x_q.device)
    _check("moe_route_topk_fp8",
           lib().moe_route_topk_fp8(_ptr(x_q), _ptr(x_d), _ptr(w_router_q), _ptr(w_router_d),
                                    _ptr(bias), T, H, N, k, n_groups, topk_groups, _ptr(scores),
                                    _ptr(idx), _ptr(gate), _ptr(ws), ws.numel(),
                                    _stream(stream)))
    return idx, gate, scores


def moe_topk_from_scores(scores, bias, k, idx=None, gate=None, n_groups=1, topk_groups=1,
                         stream=None):
    empty = _allocator(stream)
    T, N = scores.shape
    _dev(scores, torch.float32, "scores"), _dev(bias, torch.float32, "bias")
    idx = empty(T, k, dtype=torch.int32, device=scores.device) if idx is None else idx
    gate = empty(T, k, dtype=torch.float32, device=scores.device) if gate is None else gate
    _check("moe_topk_from_scores", lib().moe_topk_from_scores(
        _ptr(scores), _ptr(bias), T, N, k, n_groups, topk_groups, _ptr(idx), _ptr(gate),
        _stream(stream)))
    return idx, gate


def moe_permute_workspace_bytes(T, N, k):
    return int(lib().moe_permute_workspace_bytes(T, N, k))


def moe_permute(idx, N, with_shared=True, out=None, ws=None, stream=None):
    """idx int32 [T,k] -> (counts [N], offsets [N+2], row_of [T,k],
    token_of [T*k (+T)]), all int32."""
    empty = _allocator(stream)
    T, k = idx.shape
    _dev(idx, torch.int32, "idx")
    dev = idx.device
    if out is None:
        R = T * k + (T if with_shared else 0)
        out = (empty(N, dtype=torch.int32, device=dev),
               empty(N + 2, dtype=torch.int32, device=dev),
               empty(T, k, dtype=torch.int32, device=dev),
               empty(R, dtype=torch.int32, device=dev))
    counts, offsets, row_of, token_of = out
    nbytes = moe_permute_workspace_bytes(T, N, k)
    if ws is None:
        ws = empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _check("moe_permute", lib().moe_permute(_ptr(idx), T, N, k, 1 if with_shared else 0,
                                            _ptr(counts), _ptr(offsets), _ptr(row_of),
                                            _ptr(token_of), _ptr(ws), ws.numel(),
                                            _stream(stream)))
    return counts, offsets, row_of, token_of


def moe_permute_noalloc_max_scratch_bytes():
    return int(lib().moe_permute_noalloc_max_scratch_bytes())


def moe_permute_noalloc(idx, N, with_shared, out, stream=None):
    """moe_permute without a workspace (the library's own device scratch, for
    callers that cannot allocate): writes into the caller's ``out`` tensors
    (counts [N], offsets [N+2], row_of [T,k], token_of [T*k (+T)], int32)."""
    T, k = idx.shape
    _dev(idx, torch.int32, "idx")
    counts, offsets, row_of, token_of = out
    _check("moe_permute_noalloc", lib().moe_permute_noalloc(
        _ptr(idx), T, N, k, 1 if with_shared else 0, _ptr(counts), _ptr(offsets), _ptr(row_of),
        _ptr(token_of), _stream(stream)))
    return counts, offsets, row_of, token_of


def fp8_quant_1x128(x, q=None, d=None, stream=None):
    """x [rows, cols] bf16 or float32 -> (q uint8 [rows, cols], d float32 [rows, cols/128])."""
    empty = _allocator(stream)
    rows, cols = x.shape
    dt = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}[x.dtype]
    if x.stride(1) != 1:
        raise ValueError("x: rows must be contiguous")
    q = empty(rows, cols, dtype=torch.uint8, device=x.device) if q is None else q
    d = empty(rows, cols // 128, dtype=torch.float32, device=x.device) if d is None else d
    _check("fp8_quant_1x128", lib().fp8_quant_1x128(_ptr(x), dt, rows, cols, x.stride(0), _ptr(q),
                                                    _ptr(d), _stream(stream)))
    return q, d


def fp8_quant_128x128(w, interleave_gate_up=False, q=None, d=None, stream=None):
    """w [batch, rows, cols] bf16 -> (q uint8 like w, d float32 [batch, rows/128, cols/128])."""
    empty = _allocator(stream)
    if w.dim() == 2:
        w = w.unsqueeze(0)
    B, rows, cols = w.shape
    _dev(w, torch.bfloat16, "w")
    q = empty(B, rows, cols, dtype=torch.uint8, device=w.device) if q is None else q
    d = empty(B, rows // 128, cols // 128, dtype=torch.float32, device=w.device) \
        if d is None else d
    _check("fp8_quant_128x128", lib().fp8_quant_128x128(_ptr(w), B, rows, cols,
                                                        1 if interleave_gate_up else 0, _ptr(q),
                                                        _ptr(d), _stream(stream)))
    return q, d


def moe_grouped_gemm_fp8(a_q, a_d, b_q, b_d, group_offsets, total_rows, epilogue,
                         a_row_index=None, out=None, out_d=None, row_scale=None, stream=None,
                         tile_rows=None):
    """Grouped block-scaled FP8 GEMM (see include/moe_fp8.h).  b_q [G, n_out, K].
    tile_rows None calls moe_grouped_gemm_fp8 (the library picks the row tile);
    0, 128 or 256 calls moe_grouped_gemm_fp8_tiles with it."""
    empty = _allocator(stream)
    G, n_out, K = b_q.shape
    dev = a_q.device
    if out is None:
        if epilogue == MOE_EPI_SWIGLU_FP8:
            out = empty(total_rows, n_out // 2, dtype=torch.uint8, device=dev)
            out_d = empty(total_rows, n_out // 256, dtype=torch.float32, device=dev)
        elif epilogue == MOE_EPI_BF16:
            out = empty(total_rows, n_out, dtype=torch.bfloat16, device=dev)
        else:
            out = empty(total_rows, n_out, dtype=torch.float32, device=dev)
    args = GemmArgs(a_q.data_ptr(), a_d.data_ptr(), a_q.stride(0), a_q.shape[0],
                    a_row_index.data_ptr() if a_row_index is not None else None,
                    b_q.data_ptr(), b_d.data_ptr(), group_offsets.data_ptr(), G, total_rows,
                    n_out, K, epilogue, out.data_ptr(),
                    out_d.data_ptr() if out_d is not None else None, out.stride(0),
                    row_scale.data_ptr() if row_scale is not None else None)
    if tile_rows is None:
        _check("moe_grouped_gemm_fp8", lib().moe_grouped_gemm_fp8(ctypes.byref(args), _stream(stream)))
    else:
        _check("moe_grouped_gemm_fp8_tiles",
               lib().moe_grouped_gemm_fp8_tiles(ctypes.byref(args), int(tile_rows), _stream(stream)))
    return out, out_d


def fp8_transpose_128x128(w_q, w_d, wt_q=None, wt_d=None, stream=None):
    """Exact transpose of 128x128 block-quantised weights: w_q uint8
    [B, rows, cols], w_d float32 [B, rows/128, cols/128] -> (wt_q [B, cols,
    rows], wt_d [B, cols/128, rows/128]).  The B operand of Dgrad."""
    empty = _allocator(stream)
    if w_q.dim() == 2:
        w_q, w_d = w_q.unsqueeze(0), w_d.unsqueeze(0)
    B, rows, cols = w_q.shape
    _dev(w_q, torch.uint8, "w_q"), _dev(w_d, torch.float32, "w_d")
    dev = w_q.device
    wt_q = empty(B, cols, rows, dtype=torch.uint8, device=dev) if wt_q is None else wt_q
    wt_d = empty(B, cols // 128, rows // 128, dtype=torch.float32, device=dev) \
        if wt_d is None else wt_d
    _check("fp8_transpose_128x128", lib().fp8_transpose_128x128(
        _ptr(w_q), _ptr(w_d), B, rows, cols, _ptr(wt_q), _ptr(wt_d), _stream(stream)))
    return wt_q, wt_d


def tokens_padded_width(rows, num_groups):
    """Row stride (bytes) that holds any token-tile layout of `rows` tokens in
    `num_groups` groups: a multiple of 128, at least rows + 127 * num_groups."""
    return (rows + 127 * num_groups + 127) // 128 * 128


def fp8_quant_tokens_128(x, group_offsets, ldt=None, xt_q=None, xt_d=None, pad_offsets=None,
                         stream=None):
    """Token-tile quantiser (Wgrad operands).  x [rows, cols] bf16 or float32
    in expert-grouped row order, group_offsets int32 [G+1] -> (xt_q uint8
    [cols, ldt], xt_d float32 [cols, ldt/128], pad_offsets int32 [G+1])."""
    empty = _allocator(stream)
    rows, cols = x.shape
    G = group_offsets.numel() - 1
    dt = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}[x.dtype]
    if x.stride(1) != 1:
        raise ValueError("x: rows must be contiguous")
    _dev(group_offsets, torch.int32, "group_offsets")
    ldt = tokens_padded_width(rows, G) if ldt is None else ldt
    dev = x.device
    xt_q = empty(cols, ldt, dtype=torch.uint8, device=dev) if xt_q is None else xt_q
    xt_d = empty(cols, ldt // 128, dtype=torch.float32, device=dev) \
        if xt_d is None else xt_d
    pad_offsets = empty(G + 1, dtype=torch.int32, device=dev) if pad_offsets is None \
        else pad_offsets
    _check("fp8_quant_tokens_128", lib().fp8_quant_tokens_128(
        _ptr(x), dt, rows, cols, x.stride(0), _ptr(group_offsets), G, _ptr(xt_q), _ptr(xt_d),
        ldt, _ptr(pad_offsets), _stream(stream)))
    return xt_q, xt_d, pad_offsets


def moe_grouped_wgrad_fp8(a_q, a_d, b_q, b_d, pad_offsets, out=None, stream=None):
    """Wgrad grouped GEMM: out[g] = dY_g^T X_g (float32 [G, N, K]) from the
    token-tile operands a (dY^T, [N, lda]) and b (X^T, [K, ldb])."""
    empty = _allocator(stream)
    N, lda = a_q.shape
    K, ldb = b_q.shape
    G = pad_offsets.numel() - 1
    for t, dt, n in ((a_q, torch.uint8, "a_q"), (a_d, torch.float32, "a_d"),
                     (b_q, torch.uint8, "b_q"), (b_d, torch.float32, "b_d"),
                     (pad_offsets, torch.int32, "pad_offsets")):
        _dev(t, dt, n)
    out = empty(G, N, K, dtype=torch.float32, device=a_q.device) if out is None else out
    _check("moe_grouped_wgrad_fp8", lib().moe_grouped_wgrad_fp8(
        _ptr(a_q), _ptr(a_d), lda, N, _ptr(b_q), _ptr(b_d), ldb, K, _ptr(pad_offsets), G,
        _ptr(out), _stream(stream)))
    return out


def moe_grouped_dgrad_fp8(dy, wt_q, wt_d, group_offsets, epilogue=MOE_EPI_BF16, dy_q=None,
                          dy_d=None, out=None, stream=None):
    """Dgrad: dX = dY W per group.  dy [R, N] bf16 or float32 (grouped rows),
    wt_q/wt_d the transposed weights from fp8_transpose_128x128 ([G, K, N]).
    dY is quantised 1x128 (fp8_quant_1x128), then the grouped FP8 GEMM runs
    with the bf16 or float32 epilogue.  Returns dX [R, K]."""
    dy_q, dy_d = fp8_quant_1x128(dy, q=dy_q, d=dy_d, stream=stream)
    out, _ = moe_grouped_gemm_fp8(dy_q, dy_d, wt_q, wt_d, group_offsets, dy.shape[0], epilogue,
                                  out=out, stream=stream)
    return out


def moe_combine(out_rows, gate, row_of, shared_row0, residual=None, y=None, stream=None):
    empty = _allocator(stream)
    T, k = row_of.shape
    H = out_rows.shape[1]
    y = empty(T, H, dtype=torch.bfloat16, device=out_rows.device) if y is None else y
    _check("moe_combine", lib().moe_combine(_ptr(out_rows), _ptr(gate), _ptr(row_of), shared_row0,
                                            T, H, k, _ptr(residual), _ptr(y), _stream(stream)))
    return y


def moe_bias_update(bias, counts, T, k, gamma, stream=None):
    N = bias.shape[0]
    _check("moe_bias_update", lib().moe_bias_update(_ptr(bias), _ptr(counts), N, T, k,
                                                    float(gamma), _stream(stream)))
    return bias


def moe_seq_balance_loss(idx, gate, seq_offsets, n_experts, alpha=1e-4, loss=None, stream=None):
    """Sequence-wise balance statistic per sequence: idx int32 [T,k], gate
    float32 [T,k], seq_offsets int32 [S+1] (device) -> loss float32 [S]."""
    empty = _allocator(stream)
    T, k = idx.shape
    _dev(idx, torch.int32, "idx"), _dev(gate, torch.float32, "gate")
    _dev(seq_offsets, torch.int32, "seq_offsets")
    S = seq_offsets.numel() - 1
    loss = empty(max(S, 0), dtype=torch.float32, device=idx.device) \
        if loss is None else loss
    _check("moe_seq_balance_loss", lib().moe_seq_balance_loss(
        _ptr(idx), _ptr(gate), _ptr(seq_offsets), S, T, n_experts, k, alpha, _ptr(loss),
        _stream(stream)))
    return loss


def moe_probe_fp8_mfma(blocks, iters, sink=None, stream=None):
    """Enqueue the FP8 MFMA rate probe (a diagnostic, not a layer step):
    blocks * 4 waves, each issuing iters * 16 16x16x128 FP8 MFMAs.  Returns
    (sink, flops)."""
    if sink is None:
        sink = _allocator(stream)(blocks * 256, dtype=torch.float32, device="cuda")
    _check("moe_probe_fp8_mfma", lib().moe_probe_fp8_mfma(blocks, iters, _ptr(sink),
                                                          _stream(stream)))
    return sink, float(blocks) * 4 * iters * 16 * 65536


def moe_probe_hbm(mode, buf, sink=None, stream=None):
    """Enqueue the HBM rate probe (a diagnostic, not a layer step): modes 0
    and 2 read every byte of the device tensor ``buf`` (non-temporal, eight
    loads in flight per lane; ordinary, four), modes 1 and 3 write them
    (non-temporal; ordinary stores).  Returns the sink (read modes) or None."""
    if mode in (0, 2) and sink is None:
        sink = _allocator(stream, torch.zeros)(1, dtype=torch.int32, device=buf.device)
    _check("moe_probe_hbm", lib().moe_probe_hbm(mode, _ptr(buf), buf.numel() * buf.element_size(),
                                                _ptr(sink), _stream(stream)))
    return sink


def moe_layer_workspace_bytes(T, H, N, k, I, with_shared=True):
    return int(lib().moe_layer_workspace_bytes(T, H, N, k, I, 1 if with_shared else 0))


def moe_layer_forward(w, x, k, gamma=1e-3, n_groups=1, topk_groups=1, router_fp8=False,
                      update_bias=True, residual=None, y=None, scores=None, idx=None, gate=None,
                      counts=None, ws=None, stream=None):
    """The whole forward pass in one library call (moe_layer_forward): w a
    MoEWeights, x [T,H] bf16.  Returns y [T,H] bf16.  scores / idx / gate /
    counts: optional device outputs.  ws: optional uint8 device workspace of
    moe_layer_workspace_bytes(...) bytes (allocated here when None)."""
    empty = _allocator(stream)
    T, H = x.shape
    _dev(x, torch.bfloat16, "x"), _dev(w.bias, torch.float32, "bias")
    with_shared = w.G == w.N + 1
    if router_fp8 and w.w_router_q is None:
        raise ValueError("router_fp8 needs MoEWeights(..., router_fp8=True)")
    y = empty(T, H, dtype=torch.bfloat16, device=x.device) if y is None else y
    if ws is None:
        ws = empty(max(moe_layer_workspace_bytes(T, H, w.N, k, w.I, with_shared), 256),
                   dtype=torch.uint8, device=x.device)
    a = LayerArgs(x.data_ptr(), w.w_router.data_ptr(),
                  w.w_router_q.data_ptr() if w.w_router_q is not None else None,
                  w.w_router_d.data_ptr() if w.w_router_d is not None else None,
                  w.bias.data_ptr(), w.w1q.data_ptr(), w.w1d.data_ptr(), w.w2q.data_ptr(),
                  w.w2d.data_ptr(), T, H, w.N, k, w.I, 1 if with_shared else 0, n_groups,
                  topk_groups, 1 if router_fp8 else 0, 1 if update_bias else 0, float(gamma),
                  residual.data_ptr() if residual is not None else None, y.data_ptr(),
                  *[t.data_ptr() if t is not None else None for t in (scores, idx, gate, counts)])
    _check("moe_layer_forward", lib().moe_layer_forward(ctypes.byref(a), _ptr(ws), ws.numel(),
                                                        _stream(stream)))
    return y


# ---------------------------------------------------------------------------
# training in bf16: the norms around the block, the experts' products, the
# activation between them, and clipping


_DT = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}


def _dtype_code(t, name):
    if t.dtype not in _DT:
        raise ValueError(f"{name}: need bfloat16 or float32, got {t.dtype}")
    return _DT[t.dtype]


def _rows(t, rows, cols, dtype, name):
    """A device matrix whose rows are contiguous; returns (pointer, row stride)."""
    if t is None:
        return None, 0
    if t.dtype is dtype and t.is_cuda and t.shape == (rows, cols):
        ld, step = t.stride()
        if step == 1 or cols <= 1:
            return t.data_ptr(), ld if rows > 1 else cols
    raise ValueError(f"{name}: need a {dtype} device tensor {(rows, cols)} with contiguous "
                     f"rows, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _vector(t, n, name, dtype=torch.float32):
    if t is None:
        return None
    if t.dtype is dtype and t.is_cuda and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: need {n} contiguous {dtype} values on the device, got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _queue(stream):
    """The stream's handle (the current stream's without one)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _gate(gate, T, H, b_dtype):
    """(mode, pointer, row stride) of a gate [H], [T,1] or [T,H]."""
    if gate is None:
        return MOE_GATE_NONE, None, 0
    if gate.dim() == 1:
        return MOE_GATE_CHANNEL, _vector(gate, H, "gate"), 0
    if tuple(gate.shape) == (T, 1):
        return MOE_GATE_TOKEN, _vector(gate, T, "gate"), 0
    return (MOE_GATE_FULL, *_rows(gate, T, H, b_dtype, "gate"))


def moe_block_norm(x, b=None, w_pre=None, w_post=None, gate=None, alpha=1.0, beta=1.0, eps=1e-6,
                   r=None, h=None, stream=None):
    """The norms around a block with its gate and the residual scale:
    r = alpha x + beta gate rmsnorm(b, w_post) and h = rmsnorm(r, w_pre).
    x [T,H] the residual stream, b [T,H] the block's output (None: r is x),
    w_pre / w_post float32 [H] (None: h is not formed / b is not normalised),
    gate float32 [H] or [T,1], or [T,H] of b's type.  Returns (r, h); h has
    b's type (x's without b) unless an output is given."""
    empty = _allocator(stream)
    T, H = x.shape
    xdt = _dtype_code(x, "x")
    if b is not None:
        bt = b.dtype
        _dtype_code(b, "b")
        r = empty(T, H, dtype=x.dtype, device=x.device) if r is None else r
    else:
        if gate is not None or w_post is not None:
            raise ValueError("gate and w_post belong to a block output b")
        bt = h.dtype if h is not None else x.dtype
        r = None
    if h is None and w_pre is not None:
        h = empty(T, H, dtype=bt, device=x.device)
    mode, gp, ldg = _gate(gate, T, H, bt)
    a = BlockNormArgs(T, H, xdt, _DT.get(bt, -1), *_rows(x, T, H, x.dtype, "x"),
                      *_rows(b, T, H, bt, "b"), _vector(w_pre, H, "w_pre"),
                      _vector(w_post, H, "w_post"), mode, gp, ldg, alpha, beta, eps,
                      *_rows(r, T, H, x.dtype, "r"), *_rows(h, T, H, bt, "h"))
    _check("moe_block_norm", lib().moe_block_norm(ctypes.byref(a), _queue(stream)))
    return (x if b is None else r), h


def moe_block_norm_backward_workspace_bytes(T, H):
    return int(lib().moe_block_norm_backward_workspace_bytes(T, H))


def moe_block_norm_backward(r, dr=None, dh=None, b=None, w_pre=None, w_post=None, gate=None,
                            alpha=1.0, beta=1.0, eps=1e-6, dx=None, db=None, dw_pre=None,
                            dw_post=None, dgate=None, ws=None, stream=None):
    """Backward of moe_block_norm from r (x when there was no b) and b, given
    dr (r's other use) and dh, either of them None.  Returns (dx, db, dw_pre,
    dw_post, dgate), None where the forward pass had no such input; the
    weights' gradients and those of a [H] or [T,1] gate are float32."""
    empty = _allocator(stream)
    T, H = r.shape
    dev = r.device
    bt = b.dtype if b is not None else (dh.dtype if dh is not None else r.dtype)
    mode, gp, ldg = _gate(gate, T, H, bt)
    f32 = dict(dtype=torch.float32, device=dev)
    dx = empty(T, H, dtype=r.dtype, device=dev) if dx is None else dx
    if b is not None:
        db = empty(T, H, dtype=bt, device=dev) if db is None else db
        if w_post is not None and dw_post is None:
            dw_post = empty(H, **f32)
        if mode == MOE_GATE_FULL:
            dgate = empty(T, H, dtype=bt, device=dev) if dgate is None else dgate
        elif mode != MOE_GATE_NONE:
            dgate = empty(*gate.shape, **f32) if dgate is None else dgate
    elif gate is not None or w_post is not None:
        raise ValueError("gate and w_post belong to a block output b")
    if dh is not None and w_pre is None:
        raise ValueError("dh needs w_pre")
    if dh is not None and dw_pre is None:
        dw_pre = empty(H, **f32)
    if ws is None:
        ws = empty(max(moe_block_norm_backward_workspace_bytes(T, H), 16),
                   dtype=torch.uint8, device=dev)
    if mode == MOE_GATE_FULL:
        dgp, lddg = _rows(dgate, T, H, bt, "dgate")
    else:
        dgp, lddg = _vector(dgate, H if mode == MOE_GATE_CHANNEL else T, "dgate"), 0
    a = BlockNormBwdArgs(T, H, _dtype_code(r, "r"), _DT.get(bt, -1), *_rows(r, T, H, r.dtype, "r"),
                         *_rows(dr, T, H, r.dtype, "dr"), *_rows(dh, T, H, bt, "dh"),
                         *_rows(b, T, H, bt, "b"), _vector(w_pre, H, "w_pre"),
                         _vector(w_post, H, "w_post"), mode, gp, ldg, alpha, beta, eps,
                         *_rows(dx, T, H, r.dtype, "dx"), *_rows(db, T, H, bt, "db"),
                         _vector(dw_pre, H, "dw_pre"), _vector(dw_post, H, "dw_post"), dgp, lddg)
    _check("moe_block_norm_backward", lib().moe_block_norm_backward(
        ctypes.byref(a), _ptr(ws), ws.numel(), _queue(stream)))
    return dx, db, dw_pre, dw_post, dgate


def moe_grouped_gemm_bf16_workspace_bytes(G, total_rows, n_out, k_dim):
    return int(lib().moe_grouped_gemm_bf16_workspace_bytes(G, total_rows, n_out, k_dim))


def moe_grouped_gemm_bf16(a, b, group_offsets, total_rows, b_kn=False, a_row_index=None,
                          row_scale=None, out=None, out_dtype=torch.bfloat16, ws=None,
                          stream=None):
    """Grouped bf16 product: out[r] = row_scale[r] * A[src(r)] @ B[g]^T for the
    rows r of each group, b bf16 [G, n_out, K]; with b_kn, A[src(r)] @ B[g], b
    [G, K, n_out] (the input gradient, from the forward product's weights).
    a bf16 [rows, K] (rows contiguous), group_offsets int32 [G+1] on the
    device.  Returns out [total_rows, n_out] bf16 or float32."""
    empty = _allocator(stream)
    G = b.shape[0]
    K, n = (b.shape[1], b.shape[2]) if b_kn else (b.shape[2], b.shape[1])
    _dev(b, torch.bfloat16, "b"), _dev(group_offsets, torch.int32, "group_offsets")
    if group_offsets.numel() != G + 1:
        raise ValueError(f"group_offsets: need {G + 1} values")
    if out is None:
        out = empty(total_rows, n, dtype=out_dtype, device=a.device)
    ap, lda = _rows(a, a.shape[0], K, torch.bfloat16, "a")
    op, ldo = _rows(out, total_rows, n, out.dtype, "out")
    args = GemmBf16Args(ap, lda, a.shape[0],
                        _vector(a_row_index, total_rows, "a_row_index", torch.int32),
                        b.data_ptr(), MOE_B_KN if b_kn else MOE_B_NK, group_offsets.data_ptr(), G,
                        total_rows, n, K, _dtype_code(out, "out"), op, ldo,
                        _vector(row_scale, total_rows, "row_scale"))
    need = moe_grouped_gemm_bf16_workspace_bytes(G, total_rows, n, K)
    if ws is None and need:
        ws = empty(need, dtype=torch.uint8, device=a.device)
    _check("moe_grouped_gemm_bf16", lib().moe_grouped_gemm_bf16(
        ctypes.byref(args), _ptr(ws), ws.numel() if ws is not None else 0, _queue(stream)))
    return out


def moe_grouped_wgrad_bf16_workspace_bytes(G, total_rows, n, k):
    return int(lib().moe_grouped_wgrad_bf16_workspace_bytes(G, total_rows, n, k))


def moe_grouped_wgrad_bf16(a, b, group_offsets, total_rows, a_row_index=None, b_row_index=None,
                           accumulate=False, out=None, out_dtype=torch.float32, ws=None,
                           stream=None):
    """Weight gradients: out[g] = A_g^T B_g over the rows of each group, a bf16
    [rows, n] (the output channels' gradient), b bf16 [rows, k] (the product's
    input), each optionally gathered by its row index.  With accumulate it is
    added to out.  Returns out [G, n, k] float32 or bf16."""
    empty = _allocator(stream)
    n, k = a.shape[1], b.shape[1]
    _dev(group_offsets, torch.int32, "group_offsets")
    G = group_offsets.numel() - 1
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = empty(G, n, k, dtype=out_dtype, device=a.device)
    if tuple(out.shape) != (G, n, k):
        raise ValueError(f"out: need [{G}, {n}, {k}], got {tuple(out.shape)}")
    _dev(out, out.dtype, "out")
    ap, lda = _rows(a, a.shape[0], n, torch.bfloat16, "a")
    bp, ldb = _rows(b, b.shape[0], k, torch.bfloat16, "b")
    need = moe_grouped_wgrad_bf16_workspace_bytes(G, total_rows, n, k)
    if ws is None and need:
        ws = empty(need, dtype=torch.uint8, device=a.device)
    args = WgradBf16Args(ap, lda, a.shape[0],
                         _vector(a_row_index, total_rows, "a_row_index", torch.int32),
                         bp, ldb, b.shape[0],
                         _vector(b_row_index, total_rows, "b_row_index", torch.int32),
                         group_offsets.data_ptr(), G, total_rows, n, k, _dtype_code(out, "out"),
                         out.data_ptr(), 1 if accumulate else 0)
    _check("moe_grouped_wgrad_bf16", lib().moe_grouped_wgrad_bf16(
        ctypes.byref(args), _ptr(ws), ws.numel() if ws is not None else 0, _queue(stream)))
    return out


def moe_swiglu(a, h=None, stream=None):
    """h = silu(a[:, :I]) * a[:, I:] for rows a [R, 2I], bf16 or float32."""
    empty = _allocator(stream)
    R, I = a.shape[0], a.shape[1] // 2
    if a.shape[1] % 2:
        raise ValueError("a: need an even number of columns (gate columns, then up columns)")
    h = empty(R, I, dtype=a.dtype, device=a.device) if h is None else h
    ap, lda = _rows(a, R, 2 * I, a.dtype, "a")
    hp, ldh = _rows(h, R, I, a.dtype, "h")
    _check("moe_swiglu", lib().moe_swiglu(ap, _dtype_code(a, "a"), R, I, lda, hp, ldh,
                                          _queue(stream)))
    return h


def moe_swiglu_backward(a, dh, row_gate=None, da=None, dgate=None, hg=None, stream=None):
    """Backward of row_gate[r] * swiglu(a)[r]: a [R, 2I], dh [R, I] the gradient
    of the expert row before its gate, row_gate float32 [R] or None (all 1).
    Returns (da [R, 2I], dgate float32 [R], hg [R, I] = row_gate * swiglu(a),
    the second weight gradient's operand); pass dgate=False or hg=False for a
    result that is not wanted."""
    empty = _allocator(stream)
    R, I = dh.shape
    dt = _dtype_code(a, "a")
    da = empty(R, 2 * I, dtype=a.dtype, device=a.device) if da is None else da
    dgate = empty(R, dtype=torch.float32, device=a.device) if dgate is None else dgate
    hg = empty(R, I, dtype=a.dtype, device=a.device) if hg is None else hg
    dgate, hg = (None if t is False else t for t in (dgate, hg))
    ap, lda = _rows(a, R, 2 * I, a.dtype, "a")
    dhp, lddh = _rows(dh, R, I, a.dtype, "dh")
    dap, ldda = _rows(da, R, 2 * I, a.dtype, "da")
    hgp, ldhg = _rows(hg, R, I, a.dtype, "hg")
    _check("moe_swiglu_backward", lib().moe_swiglu_backward(
        ap, dhp, dt, R, I, lda, lddh, _vector(row_gate, R, "row_gate"), dap, ldda,
        _vector(dgate, R, "dgate"), hgp, ldhg, _queue(stream)))
    return da, dgate, hg


def _dense(t):
    """Whether the tensor's elements fill one stretch of memory, in any order."""
    if t.is_contiguous():
        return True
    order = sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1)
    at = 1
    for s, n in order:
        if s != at:
            return False
        at *= n
    return t.numel() > 0


class GradList:
    """The gradients of a model, for moe_grad_norm and moe_grad_clip: dense
    device tensors, bf16 or float32, of any sizes (a permuted view counts as
    dense).  outs: where the clipped gradients go, tensors of the same sizes
    and strides (None: in place).  Built once; valid while the tensors keep
    their memory, which this object holds on to.  Calls on one list share its
    scratch: order them on one stream.  The list may be dropped before a call
    on it has run."""

    def __init__(self, tensors, outs=None):
        tensors = list(tensors)
        outs = tensors if outs is None else list(outs)
        if len(outs) != len(tensors):
            raise ValueError("outs: need one tensor for every gradient")
        if not tensors:
            raise ValueError("tensors: need at least one gradient")
        dev = tensors[0].device
        for what, ts in (("tensors", tensors), ("outs", outs)):
            for i, t in enumerate(ts):
                _dtype_code(t, f"{what}[{i}]")
                if not t.is_cuda or t.device != dev or not _dense(t):
                    raise ValueError(f"{what}[{i}]: need a dense tensor on {dev}, got strides "
                                     f"{t.stride()} on {t.device}")
        for i, (s, d) in enumerate(zip(tensors, outs)):
            if s.shape != d.shape or (s.stride() != d.stride() and not (s.is_contiguous()
                                                                        and d.is_contiguous())):
                raise ValueError(f"outs[{i}]: need the gradient's shape and strides")
        self.tensors, self.outs, self.device = tensors, outs, dev
        self.home = _queue(None)        # the stream that table and ws belong to
        n = self.n = len(tensors)
        rows = (GradTensor * n)(*[GradTensor(s.data_ptr(), d.data_ptr(), s.numel(), _DT[s.dtype],
                                             _DT[d.dtype]) for s, d in zip(tensors, outs)])
        host = torch.empty(lib().moe_grad_table_bytes(n), dtype=torch.uint8)
        chunks = _LL(0)
        _check("moe_grad_table", lib().moe_grad_table(rows, n, host.data_ptr(), host.numel(),
                                                      ctypes.byref(chunks)))
        self.chunks = chunks.value
        self.table = host.to(dev)
        self.ws = torch.empty(lib().moe_grad_norm_workspace_bytes(self.chunks), dtype=torch.uint8,
                              device=dev)

    def _queue(self, stream):
        """The handle of a call's stream, noted with the memory that the caller
        does not see when it is not the stream which that memory belongs to."""
        queue = _queue(stream)
        if queue != self.home:
            stream = torch.cuda.current_stream() if stream is None else stream
            self.table.record_stream(stream)
            self.ws.record_stream(stream)
        return queue


def moe_grad_norm(grads, sumsq=None, norm=None, stream=None):
    """Global 2-norm of a GradList's gradients.  Returns (sumsq float64 [1],
    norm float32 [1]), both on the device."""
    empty = _allocator(stream)
    sumsq = empty(1, dtype=torch.float64, device=grads.device) if sumsq is None else sumsq
    norm = empty(1, dtype=torch.float32, device=grads.device) if norm is None else norm
    _check("moe_grad_norm", lib().moe_grad_norm(
        _ptr(grads.table), grads.n, grads.chunks, _ptr(grads.ws), grads.ws.numel(),
        _vector(sumsq, 1, "sumsq", torch.float64), _vector(norm, 1, "norm"), grads._queue(stream)))
    return sumsq, norm


def moe_grad_scale(grads, sumsq, max_norm, result=None, stream=None):
    """The scaling of moe_grad_clip from a given sum of squares (float64 [1],
    for instance summed over ranks).  Returns result float32 [2] (norm, coef)."""
    empty = _allocator(stream)
    result = empty(2, dtype=torch.float32, device=grads.device) \
        if result is None else result
    _check("moe_grad_scale", lib().moe_grad_scale(
        _ptr(grads.table), grads.n, grads.chunks, _vector(sumsq, 1, "sumsq", torch.float64),
        float(max_norm), _vector(result, 2, "result"), grads._queue(stream)))
    return result


def moe_grad_clip(grads, max_norm, result=None, stream=None):
    """Clip a GradList to max_norm: outs = coef * gradients, coef = min(1,
    max_norm / (norm + 1e-6)), or 1 when the norm is not finite.  Returns
    result float32 [2] on the device: (norm, coef)."""
    empty = _allocator(stream)
    result = empty(2, dtype=torch.float32, device=grads.device) \
        if result is None else result
    _check("moe_grad_clip", lib().moe_grad_clip(
        _ptr(grads.table), grads.n, grads.chunks, _ptr(grads.ws), grads.ws.numel(),
        float(max_norm), _vector(result, 2, "result"), grads._queue(stream)))
    return result


# ---------------------------------------------------------------------------
# the experts in microscaled 4-bit floating point


def _here(*tensors):
    """Refuses tensors of another device than the current one, whose streams
    and kernels the call would use."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
            if dev.type == "cuda" and dev.index != torch._C._cuda_getDevice():
                raise ValueError(f"need tensors on the current device, got {dev}")
        elif t.device != dev:
            raise ValueError(f"need tensors on one device, got {t.device} and {dev}")


def _counts(*sizes):
    """Refuses sizes past the 32 bits of the C entry points, which would take the
    low ones."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"need sizes below 2^31, got {max(sizes)}")


def mxfp4_code_bytes(cols):
    """Bytes of a row of codes: two columns a byte, whole blocks of 32."""
    return (cols + 31) // 32 * 16


def mxfp4_scale_bytes(cols):
    """Bytes of a row of scales: pieces of 16 for 16 blocks of columns."""
    return (cols + 511) // 512 * 16


def _matrices(x, name):
    """(dtype code, batch, rows, cols, row stride) of x [rows, cols] or [batch, rows, cols]."""
    if x.dim() not in (2, 3) or not x.is_cuda:
        raise ValueError(f"{name}: need a device tensor [rows, cols] or [batch, rows, cols], got "
                         f"{tuple(x.shape)} on {x.device}")
    batch, rows, cols = x.shape if x.dim() == 3 else (1, *x.shape)
    _counts(batch, rows, cols)
    ld = x.stride(-2) if rows > 1 else x.stride(0) if batch > 1 else max(cols, 1)
    if cols > 1 and x.stride(-1) != 1 or ld < cols or batch > 1 and x.stride(0) != rows * ld:
        raise ValueError(f"{name}: need contiguous rows at one stride, got strides {x.stride()}")
    return _dtype_code(x, name), batch, rows, cols, ld


def _packed(t, shape, name):
    """Codes or scales: uint8, dense; returns the pointer."""
    if t.dtype is torch.uint8 and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: need contiguous torch.uint8 {tuple(shape)} on the device, got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}")


def mxfp4_quant_1x32(x, values=False, interleave_gate_up=False, q=None, e=None, stream=None):
    """x [(batch,) rows, cols] bf16 or float32 in blocks of 32 columns -> (q uint8
    [..., mxfp4_code_bytes(cols)], e uint8 [..., mxfp4_scale_bytes(cols)]); with
    values (True, or a bf16 tensor to write) also what they stand for, bf16 like
    x: the third result.  interleave_gate_up: W1 = [W_gate; W_up] as the gated
    product reads it."""
    empty = _allocator(stream)
    dt, batch, rows, cols, ld = _matrices(x, "x")
    lead, dev = x.shape[:-1], x.device
    cb, sb = mxfp4_code_bytes(cols), mxfp4_scale_bytes(cols)
    q = empty(*lead, cb, dtype=torch.uint8, device=dev) if q is None else q
    e = empty(*lead, sb, dtype=torch.uint8, device=dev) if e is None else e
    if values is True:
        values = empty(*x.shape, dtype=torch.bfloat16, device=dev)
    elif values is False:
        values = None
    elif not (values.dtype is torch.bfloat16 and values.shape == x.shape and values.is_contiguous()):
        raise ValueError("values: need a contiguous bfloat16 tensor of x's shape")
    _here(x, q, e, values)
    _check("mxfp4_quant_1x32", lib().mxfp4_quant_1x32(
        x.data_ptr(), dt, batch, rows, cols, ld, 1 if interleave_gate_up else 0,
        _packed(q, (*lead, cb), "q"), _packed(e, (*lead, sb), "e"),
        None if values is None else values.data_ptr(), _queue(stream)))
    return (q, e) if values is None else (q, e, values)


def mxfp4_quant_32x1(x, q=None, e=None, stream=None):
    """The quantisation of each matrix's transpose: x [(batch,) rows, cols] bf16 or
    float32 in blocks of 32 rows -> (q uint8 [(batch,) cols, mxfp4_code_bytes(rows)],
    e uint8 [(batch,) cols, mxfp4_scale_bytes(rows)])."""
    empty = _allocator(stream)
    dt, batch, rows, cols, ld = _matrices(x, "x")
    lead = (*x.shape[:-2], cols)
    cb, sb = mxfp4_code_bytes(rows), mxfp4_scale_bytes(rows)
    q = empty(*lead, cb, dtype=torch.uint8, device=x.device) if q is None else q
    e = empty(*lead, sb, dtype=torch.uint8, device=x.device) if e is None else e
    _here(x, q, e)
    _check("mxfp4_quant_32x1", lib().mxfp4_quant_32x1(
        x.data_ptr(), dt, batch, rows, cols, ld, _packed(q, (*lead, cb), "q"),
        _packed(e, (*lead, sb), "e"), _queue(stream)))
    return q, e


def mxfp4_dequant_1x32(q, e, cols=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """What codes q [..., bytes] and scales e stand for: out [..., cols] bf16 or
    float32 (cols None: all that q has room for)."""
    empty = _allocator(stream)
    cols = 2 * q.shape[-1] if cols is None else cols
    lead = q.shape[:-1]
    rows = 1
    for n in lead:
        rows *= n
    _counts(rows, cols)
    out = empty(*lead, cols, dtype=out_dtype, device=q.device) if out is None else out
    if out.shape != (*lead, cols) or not out.is_contiguous():
        raise ValueError(f"out: need a contiguous tensor {(*lead, cols)}, got {tuple(out.shape)} "
                         f"strides {out.stride()}")
    _here(q, e, out)
    _check("mxfp4_dequant_1x32", lib().mxfp4_dequant_1x32(
        _packed(q, (*lead, mxfp4_code_bytes(cols)), "q"),
        _packed(e, (*lead, mxfp4_scale_bytes(cols)), "e"), rows, cols, _dtype_code(out, "out"),
        out.data_ptr(), cols, _queue(stream)))
    return out


def moe_grouped_gemm_mxfp4_workspace_bytes(G, total_rows, n_out, k_dim):
    return int(lib().moe_grouped_gemm_mxfp4_workspace_bytes(G, total_rows, n_out, k_dim))


def _packed_rows(t, rows, width, name):
    """Codes or scales as an operand whose rows may be strided; (pointer, stride)."""
    if t.dtype is torch.uint8 and t.is_cuda and t.dim() == 2 and t.shape == (rows, width):
        ld = t.stride(0) if rows > 1 and width else width
        if width <= 1 or t.stride(1) == 1:
            return t.data_ptr(), ld
    raise ValueError(f"{name}: need torch.uint8 {(rows, width)} with contiguous rows on the "
                     f"device, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def moe_grouped_gemm_mxfp4(a_q, a_e, b_q, b_e, group_offsets, total_rows, epilogue=None,
                           a_row_index=None, row_scale=None, out=None, out_e=None,
                           out_dtype=torch.bfloat16, k_dim=None, ws=None, stream=None):
    """Grouped product in 4-bit blocks (include/moe_fp8.h): a_q, a_e
    mxfp4_quant_1x32 of the rows, b_q [G, n_out, ...] and b_e that of the
    experts' weights.  epilogue None writes bf16 or float32 (out's type, or
    out_dtype); MOE_EPI_SWIGLU_MXFP4 the quantised gated activation.  k_dim: the
    columns (None: all that the codes have room for).  Returns (out, out_e), out_e
    None but for the gated epilogue."""
    empty = _allocator(stream)
    if b_q.dim() != 3:
        raise ValueError(f"b_q: need [G, n_out, bytes], got {tuple(b_q.shape)}")
    G, n, width = b_q.shape
    K = 2 * width if k_dim is None else k_dim
    _counts(total_rows, a_q.shape[0], n, K)
    cb, sb = mxfp4_code_bytes(K), mxfp4_scale_bytes(K)
    dev = a_q.device
    gated = epilogue == MOE_EPI_SWIGLU_MXFP4
    if gated:
        if out is None:
            out = empty(total_rows, mxfp4_code_bytes(n // 2), dtype=torch.uint8, device=dev)
        if out_e is None:
            out_e = empty(total_rows, mxfp4_scale_bytes(n // 2), dtype=torch.uint8, device=dev)
        op, ldo = _packed_rows(out, total_rows, mxfp4_code_bytes(n // 2), "out")
        oe = _packed(out_e, (total_rows, mxfp4_scale_bytes(n // 2)), "out_e")
    else:
        if out_e is not None:
            raise ValueError("out_e belongs to MOE_EPI_SWIGLU_MXFP4")
        if out is None:
            dt = torch.float32 if epilogue == MOE_EPI_F32 else out_dtype
            out = empty(total_rows, n, dtype=dt, device=dev)
        want = MOE_EPI_F32 if _dtype_code(out, "out") == MOE_F32 else MOE_EPI_BF16
        if epilogue is None:
            epilogue = want
        if epilogue != want:
            raise ValueError(f"epilogue {epilogue} does not write {out.dtype}")
        op, ldo = _rows(out, total_rows, n, out.dtype, "out")
        oe = None
    _here(a_q, a_e, b_q, b_e, group_offsets, a_row_index, row_scale, out, out_e, ws)
    ap, lda = _packed_rows(a_q, a_q.shape[0], cb, "a_q")
    ep, lde = _packed_rows(a_e, a_q.shape[0], sb, "a_e")
    args = GemmMxfp4Args(ap, lda, ep, lde, a_q.shape[0],
                         _vector(a_row_index, total_rows, "a_row_index", torch.int32),
                         _packed(b_q, (G, n, cb), "b_q"), _packed(b_e, (G, n, sb), "b_e"),
                         _vector(group_offsets, G + 1, "group_offsets", torch.int32), G, total_rows,
                         n, K, epilogue, op, ldo, oe, _vector(row_scale, total_rows, "row_scale"))
    need = moe_grouped_gemm_mxfp4_workspace_bytes(G, total_rows, n, K)
    if ws is None and need:
        ws = empty(need, dtype=torch.uint8, device=dev)
    _check("moe_grouped_gemm_mxfp4", lib().moe_grouped_gemm_mxfp4(
        ctypes.byref(args), _ptr(ws), ws.numel() if ws is not None else 0, _queue(stream)))
    return out, out_e


def moe_grouped_dgrad_mxfp4(dy, wt_q, wt_e, group_offsets, out=None, out_dtype=torch.bfloat16,
                            ws=None, stream=None):
    """Input gradient dX = dY W per group in 4-bit blocks: dy [R, N] bf16 or float32
    (grouped rows), wt_q / wt_e the turned weights of mxfp4_quant_32x1 ([G, K, ...]).
    Returns dX [R, K]."""
    dy_q, dy_e = mxfp4_quant_1x32(dy, stream=stream)
    return moe_grouped_gemm_mxfp4(dy_q, dy_e, wt_q, wt_e, group_offsets, dy.shape[0], out=out,
                                  out_dtype=out_dtype, k_dim=dy.shape[1], ws=ws, stream=stream)[0]


# ---------------------------------------------------------------------------
# the router's balance loss for training


class BalanceStats:
    """What moe_balance_loss leaves of the sequences: load and prob float32 [S, N],
    counts int32 [S, N] (the experts' picks), tokens int32 [S]."""

    def __init__(self, load, prob, counts, tokens):
        self.load, self.prob, self.counts, self.tokens = load, prob, counts, tokens


def moe_balance_loss_workspace_bytes(T, N, n_seq):
    return int(lib().moe_balance_loss_workspace_bytes(T, N, n_seq))


def _sequences(seq_offsets, token_mask, T):
    """(count, offsets' pointer, mask's pointer)."""
    mp = None
    if token_mask is not None:
        if token_mask.dtype is torch.bool:
            token_mask = token_mask.view(torch.uint8)
        mp = _vector(token_mask, T, "token_mask", torch.uint8)
    if seq_offsets is None:
        return 1, None, mp
    n = seq_offsets.numel()
    if n < 1:
        raise ValueError("seq_offsets: need at least one value")
    return n - 1, _vector(seq_offsets, n, "seq_offsets", torch.int32), mp


def moe_balance_loss(scores, idx, seq_offsets=None, token_mask=None, alpha=1e-4, loss=None,
                     stats=None, ws=None, stream=None):
    """The router's balance loss of each sequence (include/moe_fp8.h): scores
    float32 [T, N] and idx int32 [T, k] as the router writes them, seq_offsets
    int32 [S+1] on the device (None: one sequence of all tokens), token_mask bool
    or uint8 [T] (None: every token counts).  Returns (loss float32 [S],
    BalanceStats), which moe_router_backward takes."""
    empty = _allocator(stream)
    T, N = scores.shape
    dev, k = scores.device, idx.shape[1]
    S, sp, mp = _sequences(seq_offsets, token_mask, T)
    _counts(T, N, k, S)
    loss = empty(S, dtype=torch.float32, device=dev) if loss is None else loss
    if stats is None:
        stats = BalanceStats(empty(S, N, dtype=torch.float32, device=dev),
                             empty(S, N, dtype=torch.float32, device=dev),
                             empty(S, N, dtype=torch.int32, device=dev),
                             empty(S, dtype=torch.int32, device=dev))
    need = moe_balance_loss_workspace_bytes(T, N, S)
    if ws is None and need:
        ws = empty(need, dtype=torch.uint8, device=dev)
    _here(scores, idx, seq_offsets, token_mask, loss, stats.load, stats.prob, stats.counts,
          stats.tokens, ws)
    sc, lds = _rows(scores, T, N, torch.float32, "scores")
    a = BalanceArgs(T, N, k, S, sc, max(lds, N), _vector(idx, T * k, "idx", torch.int32), sp, mp,
                    alpha, _vector(loss, S, "loss"), _vector(stats.load, S * N, "load"),
                    _vector(stats.prob, S * N, "prob"),
                    _vector(stats.counts, S * N, "counts", torch.int32),
                    _vector(stats.tokens, S, "tokens", torch.int32))
    _check("moe_balance_loss", lib().moe_balance_loss(
        ctypes.byref(a), _ptr(ws), ws.numel() if ws is not None else 0, _queue(stream)))
    return loss, stats


def moe_router_backward(scores, idx, gate=None, dgate=None, load=None, tokens=None,
                        seq_offsets=None, token_mask=None, dloss=None, alpha=1e-4, dz=None,
                        out_dtype=torch.bfloat16, stream=None):
    """Gradient dz [T, N] (bf16 or float32) of the router's logits: from dgate
    float32 [T, k], that of the gates (None: left out), and from the balance loss
    with the load [S, N] and tokens [S] of its BalanceStats (None: left out),
    dloss float32 [S] being its gradient (None: 1).  Other arguments as
    moe_balance_loss took them."""
    empty = _allocator(stream)
    T, N = scores.shape
    k = idx.shape[1]
    if dgate is not None and gate is None:
        raise ValueError("dgate needs gate")
    if load is not None and tokens is None:
        raise ValueError("load needs tokens")
    S, sp, mp = _sequences(seq_offsets, token_mask, T)
    _counts(T, N, k, S)
    dz = empty(T, N, dtype=out_dtype, device=scores.device) if dz is None else dz
    _here(scores, idx, gate, dgate, load, tokens, seq_offsets, token_mask, dloss, dz)
    sc, lds = _rows(scores, T, N, torch.float32, "scores")
    zp, ldz = _rows(dz, T, N, dz.dtype, "dz")
    a = RouterBwdArgs(T, N, k, S, sc, lds, _vector(idx, T * k, "idx", torch.int32),
                      _vector(gate, T * k, "gate"), _vector(dgate, T * k, "dgate"),
                      _vector(load, S * N, "load"), _vector(tokens, S, "tokens", torch.int32), sp,
                      mp, _vector(dloss, S, "dloss"), alpha, _dtype_code(dz, "dz"), zp, ldz)
    _check("moe_router_backward", lib().moe_router_backward(ctypes.byref(a), _queue(stream)))
    return dz


# ---------------------------------------------------------------------------
# the layer


class MoEWeights:
    """Device weights of one layer: router [N,H] bf16, bias [N] float32, and
    FP8 experts quantised 128x128 from bf16 W1 [G,2I,H] (gate rows, then up
    rows) and W2 [G,H,I]; expert G-1 = N is the shared expert.  router_fp8
    also keeps the router quantised 128x128 for the opt-in FP8 router."""

    def __init__(self, w_router, bias, w1_bf16=None, w2_bf16=None, w1q=None, w1d=None,
                 w2q=None, w2d=None, router_fp8=False):
        self.w_router = w_router
        self.bias = bias
        self.w_router_q = self.w_router_d = None
        if router_fp8:   # the opt-in FP8 router: Wr quantised 128x128 as well
            q, d = fp8_quant_128x128(w_router)
            self.w_router_q, self.w_router_d = q[0], d[0]
        if w1_bf16 is not None:
            w1q, w1d = fp8_quant_128x128(w1_bf16, interleave_gate_up=True)
        if w2_bf16 is not None:
            w2q, w2d = fp8_quant_128x128(w2_bf16)
        self.w1q, self.w1d, self.w2q, self.w2d = w1q, w1d, w2q, w2d
        self.N, self.H = w_router.shape
        self.G = w1q.shape[0]
        self.I = w1q.shape[1] // 2


class MoELayer:
    """Buffers for a batch of T tokens and the forward pass over them.  All
    buffers are allocated once here; ``forward`` only enqueues kernels."""

    def __init__(self, weights, T, k, gamma=1e-3, device="cuda", n_groups=1, topk_groups=1,
                 router_fp8=False):
        w = weights
        self.w, self.T, self.k, self.gamma = w, T, k, gamma
        self.n_groups, self.topk_groups = n_groups, topk_groups
        if router_fp8 and w.w_router_q is None:
            raise ValueError("router_fp8 needs MoEWeights(..., router_fp8=True)")
        self.router_fp8 = router_fp8
        N, H, I = w.N, w.H, w.I
        self.with_shared = w.G == N + 1
        R = T * k + (T if self.with_shared else 0)
        self.R = R
        e = dict(device=device)
        self.scores = torch.empty(T, N, dtype=torch.float32, **e)
        self.idx = torch.empty(T, k, dtype=torch.int32, **e)
        self.gate = torch.empty(T, k, dtype=torch.float32, **e)
        self.counts = torch.empty(N, dtype=torch.int32, **e)
        self.offsets = torch.empty(N + 2, dtype=torch.int32, **e)
        self.row_of = torch.empty(T, k, dtype=torch.int32, **e)
        self.token_of = torch.empty(R, dtype=torch.int32, **e)
        self.ws = torch.empty(max(moe_permute_workspace_bytes(T, N, k), 16), dtype=torch.uint8, **e)
        self.route_ws = torch.empty(max(moe_route_workspace_bytes(T, H, N), 16), dtype=torch.uint8,
                                    **e)
        self._operands(e)
        self.out_rows = torch.empty(R, H, dtype=torch.bfloat16, **e)
        self.y = torch.empty(T, H, dtype=torch.bfloat16, **e)

    def _operands(self, e):
        """The products' quantised operands."""
        T, R, H, I = self.T, self.R, self.w.H, self.w.I
        self.xq = torch.empty(T, H, dtype=torch.uint8, **e)
        self.xd = torch.empty(T, H // 128, dtype=torch.float32, **e)
        self.hq = torch.empty(R, I, dtype=torch.uint8, **e)
        self.hd = torch.empty(R, I // 128, dtype=torch.float32, **e)

    # the individual steps, so that callers can time or replace one of them
    def route(self, x, stream=None):
        """Routing from x with the bf16 router, which also writes the 1x128
        quantisation of x into self.xq / self.xd from the same read of x; or,
        with the FP8 router, from the quantised x already there (quant_x runs
        first)."""
        if self.router_fp8:
            moe_route_topk_fp8(self.xq, self.xd, self.w.w_router_q, self.w.w_router_d,
                               self.w.bias, self.k, scores=self.scores, idx=self.idx,
                               gate=self.gate, ws=self.route_ws, n_groups=self.n_groups,
                               topk_groups=self.topk_groups, stream=stream)
            return
        moe_route_topk_quant_x(x, self.w.w_router, self.w.bias, self.k, x_q=self.xq, x_d=self.xd,
                               scores=self.scores, idx=self.idx, gate=self.gate,
                               ws=self.route_ws, n_groups=self.n_groups,
                               topk_groups=self.topk_groups, stream=stream)

    def permute(self, stream=None):
        moe_permute(self.idx, self.w.N, self.with_shared,
                    out=(self.counts, self.offsets, self.row_of, self.token_of), ws=self.ws,
                    stream=stream)

    def quant_x(self, x, stream=None):
        fp8_quant_1x128(x, q=self.xq, d=self.xd, stream=stream)

    def gemm1(self, stream=None):
        moe_grouped_gemm_fp8(self.xq, self.xd, self.w.w1q, self.w.w1d, self.offsets, self.R,
                             MOE_EPI_SWIGLU_FP8,
                             a_row_index=self.token_of, out=self.hq, out_d=self.hd, stream=stream)

    def gemm2(self, stream=None):
        moe_grouped_gemm_fp8(self.hq, self.hd, self.w.w2q, self.w.w2d, self.offsets, self.R,
                             MOE_EPI_BF16, out=self.out_rows, stream=stream)

    def combine(self, stream=None):
        moe_combine(self.out_rows, self.gate, self.row_of,
                    self.T * self.k if self.with_shared else -1, y=self.y, stream=stream)

    def bias_update(self, stream=None):
        moe_bias_update(self.w.bias, self.counts, self.T, self.k, self.gamma, stream=stream)

    def forward(self, x, update_bias=True, stream=None):
        """One forward pass of the layer over x [T,H] bf16; returns y [T,H]
        bf16 (a buffer of this object).  With update_bias the per-expert bias
        is updated from this batch's counts at the end."""
        if self.router_fp8:
            self.quant_x(x, stream)
        self.route(x, stream)
        self.permute(stream)
        self.gemm1(stream)
        self.gemm2(stream)
        self.combine(stream)
        if update_bias:
            self.bias_update(stream)
        return self.y


class MoEWeightsMxfp4:
    """Device weights of one layer whose experts are in 4-bit blocks: router [N,H]
    bf16, bias [N] float32, and the experts quantised by mxfp4_quant_1x32 from bf16
    W1 [G,2I,H] (gate rows, then up rows; interleaved in blocks of 128) and W2
    [G,H,I], or given so; expert G-1 = N is the shared expert."""

    def __init__(self, w_router, bias, w1_bf16=None, w2_bf16=None, w1q=None, w1e=None,
                 w2q=None, w2e=None):
        self.w_router, self.bias = w_router, bias
        self.w_router_q = None
        if w1_bf16 is not None:
            w1q, w1e = mxfp4_quant_1x32(w1_bf16, interleave_gate_up=True)
        if w2_bf16 is not None:
            w2q, w2e = mxfp4_quant_1x32(w2_bf16)
        self.w1q, self.w1e, self.w2q, self.w2e = w1q, w1e, w2q, w2e
        self.N, self.H = w_router.shape
        self.G = w1q.shape[0]
        self.I = w1q.shape[1] // 2


class MoELayerMxfp4(MoELayer):
    """MoELayer with the experts in 4-bit blocks (MoEWeightsMxfp4): the same routing,
    permutation, combine and bias update around two products whose operands are
    4-bit codes, activations included.  Requires I % 128 == 0."""

    def __init__(self, weights, T, k, gamma=1e-3, device="cuda", n_groups=1, topk_groups=1):
        if weights.I % 128:
            raise ValueError(f"the expert width must be a multiple of 128, got {weights.I}")
        super().__init__(weights, T, k, gamma, device, n_groups, topk_groups)

    def _operands(self, e):
        w, T, R = self.w, self.T, self.R
        u8 = dict(dtype=torch.uint8, **e)
        self.xq = torch.empty(T, mxfp4_code_bytes(w.H), **u8)
        self.xe = torch.empty(T, mxfp4_scale_bytes(w.H), **u8)
        self.hq = torch.empty(R, mxfp4_code_bytes(w.I), **u8)
        self.he = torch.empty(R, mxfp4_scale_bytes(w.I), **u8)
        need = max(moe_grouped_gemm_mxfp4_workspace_bytes(w.G, R, 2 * w.I, w.H),
                   moe_grouped_gemm_mxfp4_workspace_bytes(w.G, R, w.H, w.I))
        self.gemm_ws = torch.empty(max(need, 16), **u8)

    def route(self, x, stream=None):
        """Routing from x, and x quantised into self.xq / self.xe."""
        moe_route_topk(x, self.w.w_router, self.w.bias, self.k, scores=self.scores, idx=self.idx,
                       gate=self.gate, ws=self.route_ws, n_groups=self.n_groups,
                       topk_groups=self.topk_groups, stream=stream)
        self.quant_x(x, stream)

    def quant_x(self, x, stream=None):
        mxfp4_quant_1x32(x, q=self.xq, e=self.xe, stream=stream)

    def gemm1(self, stream=None):
        moe_grouped_gemm_mxfp4(self.xq, self.xe, self.w.w1q, self.w.w1e, self.offsets[:self.w.G + 1],
                               self.R, MOE_EPI_SWIGLU_MXFP4, a_row_index=self.token_of, out=self.hq,
                               out_e=self.he, k_dim=self.w.H, ws=self.gemm_ws, stream=stream)

    def gemm2(self, stream=None):
        moe_grouped_gemm_mxfp4(self.hq, self.he, self.w.w2q, self.w.w2e, self.offsets[:self.w.G + 1],
                               self.R, out=self.out_rows, k_dim=self.w.I, ws=self.gemm_ws,
                               stream=stream)
