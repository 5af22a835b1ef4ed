"""The layer with its experts in 4-bit blocks at batches whose products run in row tiles taken
from the counters of the workspace that both products share: sampled rows of every step
against float64 on the step's own inputs, and captured and replayed.  Bars as in
``test_gpu_layer_mx``."""
import numpy as np
import pytest

from helpers import log
from oracle import mx
from test_gpu_layer_mx import _layer, _values
from test_gpu_mx import _bar, _check_h, _want

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


def _in_row_tiles(moe, layer):
    """Both products take more tiles than there are workgroups, with different needs."""
    w = layer.w
    assert layer.R > 64 * w.G
    for n, k in ((2 * w.I, w.H), (w.H, w.I)):
        need = moe.moe_grouped_gemm_mxfp4_workspace_bytes(w.G, layer.R, n, k)
        assert 0 < need <= layer.gemm_ws.numel()


@pytest.mark.parametrize("T,H,I,N,k", [(1100, 7168, 2048, 32, 2), (1301, 1664, 896, 16, 3)])
def test_prefill_in_row_tiles(moe, T, H, I, N, k):
    layer, x, w1, w2 = _layer(moe, T, H, I, N, k, seed=T)
    _in_row_tiles(moe, layer)
    layer.gemm_ws.fill_(255)
    log(f"MoELayerMxfp4 in row tiles T={T} H={H} I={I} N={N} k={k}")
    y = _values(layer.forward(x))
    off, token_of = layer.offsets.cpu().numpy(), layer.token_of.cpu().numpy()
    order = mx.interleave(2 * I)
    sizes = np.diff(off[:N + 2])
    assert sizes[N] == T
    pair = lambda v: [v.reshape(len(v), -1, 2, 128)[:, :, i].reshape(len(v), I) for i in (0, 1)]  # noqa: E731
    # the largest and the smallest routed expert, and the shared one, whose tiles have up to 288 rows
    routed = np.flatnonzero(sizes[:N])
    for e in {int(routed[np.argmax(sizes[routed])]), int(routed[np.argmin(sizes[routed])]), N}:
        rows = np.unique(np.linspace(off[e], off[e + 1] - 1, 60).astype(int))
        at = torch.from_numpy(rows).cuda()
        xv = _want(_values(x[torch.from_numpy(token_of[rows]).long().cuda()]))[2]
        C, mag = mx.grouped_gemm(xv, _want(_values(w1[e])[order])[2][None], [0, len(rows)])
        h = mx.gated(C)
        (g, u), (dg, du) = pair(C), pair(((H + 127) // 128 * 4) * 2.0 ** -24 * mag)
        tol = 1.1 * np.abs(u) * dg + np.abs(g / (1 + np.exp(-g))) * du + (16 + 2 * np.abs(g)) * 2.0 ** -24 * np.abs(h)
        hq, he = layer.hq[at].cpu().numpy(), layer.he[at].cpu().numpy()
        assert _check_h(hq, he, h, tol) <= 1e-3
        out, mag = mx.grouped_gemm(mx.values(*mx.unpack(hq, he), I), _want(_values(w2[e]))[2][None], [0, len(rows)])
        got = _values(layer.out_rows[at])
        assert np.all(np.abs(got - out) <= _bar(out, mag, I, "bf16"))
    row_of, gates = layer.row_of.long(), layer.gate.double()
    for t in (0, 1, T // 2, T - 1):
        rows = _values(layer.out_rows[row_of[t]])
        terms = np.concatenate([gates[t].cpu().numpy()[:, None] * rows, _values(layer.out_rows[T * k + t])[None]])
        want, size = terms.sum(0), np.abs(terms).sum(0)
        assert np.all(np.abs(y[t] - want) <= 2.0 ** -8 * np.abs(want) + (k + 1) * 2.0 ** -24 * size)


def test_prefill_captured_and_replayed(moe):
    """A captured layer whose products share counters, replayed on new inputs with eager work
    of the same layer between the replays."""
    shape = (1301, 1664, 896, 16, 3)
    layer, x, _, _ = _layer(moe, *shape, seed=5)
    twin, _, _, _ = _layer(moe, *shape, seed=5)
    _in_row_tiles(moe, layer)
    layer.forward(x, update_bias=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(x)
    for step in range(4):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(step))
        log(f"MoELayerMxfp4 in row tiles, replay {step}")
        y.zero_()
        graph.replay()
        first = y.clone()
        want = twin.forward(x.clone())
        torch.cuda.synchronize()
        assert torch.equal(first, want) and torch.equal(layer.w.bias, twin.w.bias)
        again = layer.forward(x, update_bias=False)       # eagerly, on the same buffers
        want = twin.forward(x.clone(), update_bias=False)
        torch.cuda.synchronize()
        assert torch.equal(again, want)
